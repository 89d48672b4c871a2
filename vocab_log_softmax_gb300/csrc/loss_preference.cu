// Preference loss of paired sequences: the row kernel's log-probability form,
// the pair kernel, the weighted sum of any loss's terms, and the gradient
// from saved statistics.
#include "loss_rows.cuh"

namespace vls {

namespace {

constexpr int kPairThreads = 1024;

// log(1 + e^x)
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Sum of an integer over the CTA.
__device__ __forceinline__ int block_count(int n) {
  __shared__ int total;
  __syncthreads();
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) atomicAdd(&total, n);   // integers: any order gives the same
  __syncthreads();
  return total;
}

// One CTA per pair: R_s = sum over the rows of sequence s with a target of
// (logp - ref), in two floats because a long answer's sum is hundreds of times
// the difference that matters; u = beta (R_chosen - R_rejected) - margin, its loss
// and the coefficient dL/dlogp of every row of the two sequences.  The last
// CTA gives the rows that no sequence holds the coefficient and statistics of a
// row without a target, so that whatever their logits hold reaches no gradient.
// Bound by
// latency (two dependent sweeps of 20 bytes a row): a few us beside the launches
// over the logits, hidden in part by the dependent launch (3 launches over 64 x
// 32000 bf16 in 10.5 us).
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const PairArgs a) {
  __shared__ Sum2 buf[2][kPairThreads / 32];
  __shared__ float s_g[2];
  dependents_may_launch();
  wait_for_previous();
  const int64_t P = a.pairs;
  auto clip_row = [&](int64_t r) { return r < 0 ? 0 : (r > a.rows ? a.rows : r); };
  if (blockIdx.x == P) {
    const int64_t first = clip_row(a.offsets[0]), last = clip_row(a.offsets[2 * P]);
    auto clear = [&](int64_t r) {
      a.coef[r] = 0.0f;
      a.stats[r] = vls_rowstat{0.0f, 0.0f};
    };
    for (int64_t r = threadIdx.x; r < first; r += kPairThreads) clear(r);
    for (int64_t r = last + threadIdx.x; r < a.rows; r += kPairThreads) clear(r);
    return;
  }
  const int64_t pair = blockIdx.x;
  Sum2 total[2];
  float per[2];
  int64_t beg[2], end[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int64_t s = pair + side * P;
    beg[side] = clip_row(a.offsets[s]);
    end[side] = clip_row(a.offsets[s + 1]);
    Sum2 sum{0.0f, 0.0f};
    int count = 0;
#pragma unroll 4
    for (int64_t r = beg[side] + threadIdx.x; r < end[side]; r += kPairThreads) {
      if (!dev::valid_id(a.ids[r], a.vocab, a.ignore_index)) continue;
      sum.add(a.logp[r]);
      if (a.ref_logp != nullptr) sum.add(-a.ref_logp[r]);
      ++count;
    }
    per[side] = 1.0f;
    if (a.average) {
      count = block_count(count);
      per[side] = 1.0f / static_cast<float>(count > 1 ? count : 1);
    }
    total[side] = cta_sum(sum, buf[side]);
  }
  if (threadIdx.x == 0) {
    // the scaled sums; without averaging their difference keeps both parts
    const float beta = a.beta;
    const float r0 = total[0].value() * per[0], r1 = total[1].value() * per[1];
    float diff = r0 - r1;
    if (!a.average) {
      Sum2 d = total[0];
      d.add(Sum2{-total[1].hi, -total[1].lo});
      diff = d.value();
    }
    const float u = beta * diff - (a.margin != nullptr ? a.margin[pair] : 0.0f);
    float loss, du;
    if (a.kind == VLS_PREF_SIGMOID) {
      const float l = a.label_smoothing;
      loss = (1.0f - l) * softplus(-u) + (l > 0.0f ? l * softplus(u) : 0.0f);
      du = -(1.0f - l) * sigmoid(-u) + (l > 0.0f ? l * sigmoid(u) : 0.0f);
      if (isnan(u)) loss = u;
    } else if (a.kind == VLS_PREF_HINGE) {
      loss = u < 1.0f ? 1.0f - u : (isnan(u) ? u : 0.0f);
      du = u < 1.0f ? -1.0f : (isnan(u) ? u : 0.0f);
    } else {
      const float e = (u - 0.5f) / beta;   // (u / beta - 1 / (2 beta))^2
      loss = e * e;
      du = 2.0f * e / beta;
    }
    const float w = a.weights != nullptr ? a.weights[pair] : 1.0f;
    a.pair_loss[pair] = loss;
    a.reward[pair] = beta * r0;
    a.reward[pair + P] = beta * r1;
    s_g[0] = beta * du * w * per[0];
    s_g[1] = -beta * du * w * per[1];
  }
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const float g = s_g[side];
#pragma unroll 4
    for (int64_t r = beg[side] + threadIdx.x; r < end[side]; r += kPairThreads)
      a.coef[r] = dev::valid_id(a.ids[r], a.vocab, a.ignore_index) ? g : 0.0f;
  }
}

constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads) loss_sum_kernel(const float* v, const float* w, int64_t n, float* out) {
  wait_for_previous();
  weighted_sum(v, w, n, out);
}

template <class T, bool CAP, bool TOPK>
cudaError_t launch_grad_k(const LossGradArgs& a, bool follows, cudaStream_t s) {
  const size_t smem = TOPK ? target_smem(a.k) : 0;
  const unsigned grid = static_cast<unsigned>(a.rows * a.chunks + (a.sum_out != nullptr ? 1 : 0));
  const auto kernel = rows_aligned<T>(a.x, a.rx, a.dx, a.vocab) ? loss_grad_kernel<T, CAP, true, TOPK>
                                                                 : loss_grad_kernel<T, CAP, false, TOPK>;
  if (follows) return launch_dependent(kernel, grid, kLossThreads, smem, s, a);
  kernel<<<grid, kLossThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <class T, bool CAP>
cudaError_t launch_grad_t(const LossGradArgs& a, bool follows, cudaStream_t s) {
  return a.k > 1 ? launch_grad_k<T, CAP, true>(a, follows, s) : launch_grad_k<T, CAP, false>(a, follows, s);
}

}  // namespace

cudaError_t launch_loss_logp(vls_dtype dt, bool cap, const LossArgs& a, cudaStream_t s) {
  return launch_loss_op<kLossLogp>(dt, cap, a, s);
}

cudaError_t launch_loss_pairs(const PairArgs& a, bool follows, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.pairs + 1);
  if (follows) return launch_dependent(pair_kernel, grid, kPairThreads, 0, s, a);
  pair_kernel<<<grid, kPairThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_loss_sum(const float* v, const float* w, int64_t n, float* out, cudaStream_t s) {
  return launch_dependent(loss_sum_kernel, 1u, kSumThreads, 0, s, v, w, n, out);
}

cudaError_t launch_loss_grad(vls_dtype dt, bool cap, const LossGradArgs& a, bool follows, cudaStream_t s) {
  if (dt == VLS_BF16)
    return cap ? launch_grad_t<__nv_bfloat16, true>(a, follows, s) : launch_grad_t<__nv_bfloat16, false>(a, follows, s);
  if (dt == VLS_F16) return cap ? launch_grad_t<__half, true>(a, follows, s) : launch_grad_t<__half, false>(a, follows, s);
  return cap ? launch_grad_t<float, true>(a, follows, s) : launch_grad_t<float, false>(a, follows, s);
}

}  // namespace vls
