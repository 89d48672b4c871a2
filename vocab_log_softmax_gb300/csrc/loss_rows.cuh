// Training losses of a row's target log-probabilities, with the gradient of
// the logits from the same launch.
//
// Every loss here is, per row, a function of the log-probabilities
//   log q_j = log_softmax(z / tau)[id_j],  z = x or cap * tanh(x / cap),
// of the row's k target ids, so with c_j = w dL/dlog q_j its gradient is
//   dL/dx = (sum_j c_j onehot(id_j) - G q) (dz/dx) / tau,   G = sum_j c_j.
// A row's gradient needs the row's own statistics only, so one launch can
// sweep the row (max and sum of exponentials), form the loss and write the
// gradient: the logits cross HBM once, against twice for a statistics launch
// followed by a gradient launch.
//
// Launch shape: a cluster of `cluster` CTAs per row, a function of V and the
// dtype only; each CTA owns a contiguous run of columns, thread t of
// kLossThreads the units (kCols columns) t, t + kLossThreads, ... of that run.
// Reduction order: the columns of a unit, the thread's units in increasing order,
// lanes xor 16..1, warps xor 4..1, cluster ranks xor 8..1.  Nothing depends on N,
// on the row's position or on its alignment.
#pragma once

#include <atomic>

#include "vls_device.cuh"

namespace vls {

using namespace dev;

// Programmatic dependent launch: a kernel of a call that follows another one of
// the same call is launched while that one still runs (dependents_may_launch)
// and waits for its end, and its memory, before it touches anything
// (wait_for_previous; nothing to wait for without the launch attribute).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class K, class... A>
cudaError_t launch_dependent(K kernel, unsigned grid, unsigned block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Temperature and softcap of a row's logits.  Weights are powers of two:
// (z - m) kk with kk = log2(e) / tau.  With a cap the weight's exponent is
// a2 r + b2 (vls_device.cuh), both terms scaled by 1 / tau.
struct Scale {
  float kk, inv_tau;
  CapK K;
};
__device__ __forceinline__ Scale make_scale(float cap, float inv_tau) {
  Scale s;
  s.inv_tau = inv_tau;
  s.kk = kLog2e * inv_tau;
  s.K = cap_consts(cap > 0.0f ? cap : 1.0f);
  s.K.a2 *= inv_tau;
  return s;
}

// The centre of a sum whose max is m: 0 when nothing finite has been seen, so
// that -inf columns weigh 0 and a NaN column still makes the sum NaN.
__device__ __forceinline__ float centre(float m) { return m > neg_inf() ? m : 0.0f; }

// Max (of x, or with a cap of z) and the sum of 2^((z - m) kk) over part of a row.
struct MaxSum {
  float m, s;
};
// Combines the parts that lanes 0..W-1 of a warp hold (lanes from `n` on hold
// none); every one of those lanes gets the result.  Order: xor W/2, ..., 1.
template <int W>
__device__ __forceinline__ MaxSum merge_lanes(MaxSum p, int n, float kk) {
  const bool on = static_cast<int>(threadIdx.x & 31) < n;
  const float M = warp_max(on ? p.m : neg_inf());
  float s = on ? p.s * ex2((p.m - centre(M)) * kk) : 0.0f;
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return {M, s};
}

// log S = e ln 2 + log f with S = 2^e f, 1 <= f < 2, kept apart: log-probabilities
// subtract the two parts one after the other, which leaves the rounding of a
// number near the result instead of that of log S.
struct LogSum {
  float e, lf;
  __device__ __forceinline__ float sub_from(float d) const { return fmaf(-e, kLn2, d) - lf; }
  __device__ __forceinline__ float value() const { return fmaf(e, kLn2, lf); }
};
__device__ __forceinline__ LogSum log_sum(float S) {
  const uint32_t b = __float_as_uint(S);
  if (!(S < pos_inf()) || b < 0x00800000u) return {0.0f, logf(S)};   // NaN, inf, subnormal
  return {static_cast<float>(static_cast<int>(b >> 23) - 127), logf(__uint_as_float((b & 0x007fffffu) | 0x3f800000u))};
}

// The columns a thread handles at a time: one 16-byte granule, 8 columns of a
// 16-bit type (Raw8) or 4 of fp32 (Raw4; with 8, neighbouring threads' shared
// memory reads lie 32 bytes apart and meet in the same banks).
struct Raw4 {
  float v[4];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = ld_stream16(p);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
  }
  // columns j >= valid read as -inf
  __device__ __forceinline__ void load_scalar(const float* p, int valid) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < valid ? __ldg(p + j) : neg_inf();
  }
  __device__ __forceinline__ float max() const { return fmaxf(max3(v[0], v[1], v[2]), v[3]); }
  __device__ __forceinline__ fp2 pair(int i) const { return pk(v[2 * i], v[2 * i + 1]); }
};
__device__ __forceinline__ fp2 pair_min(const Raw4& x, int i, const CapK& K) {
  return pk(min_nan(x.v[2 * i], K.xmax), min_nan(x.v[2 * i + 1], K.xmax));
}
template <class T>
using Unit = std::conditional_t<sizeof(T) == 4, Raw4, Raw8<T>>;
template <class T>
constexpr int kCols = sizeof(T) == 4 ? 4 : 8;
template <class T>
constexpr int kPairs = kCols<T> / 2;

template <class T>
__device__ __forceinline__ void store_unit(T* p, const fp2 (&o)[kPairs<T>]) {
  if constexpr (sizeof(T) == 4) {
    float a, b, c, d;
    upk(o[0], a, b);
    upk(o[1], c, d);
    st16(p, make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)));
  } else {
    Out8<T>::store(p, o);
  }
}

// The softcapped weight's exponent and the gradient's r of pair i of a unit, as
// cap_d2_pair and cap_r_pair (vls_device.cuh) form them; the reciprocal's form
// depends on the pair's place in the unit.
template <class U>
__device__ __forceinline__ fp2 cap_weight(const U& v, int i, const CapK& K, fp2 b2) {
  fp2 r;
  if ((kCapFmaPairs >> i) & 1u)
    r = rcp2_fma_neg(sub2(splat(-1.0f), ex2_2(mul2(pair_min(v, i, K), splat(K.k2)))));
  else
    r = rcp2(add2(ex2_2(mul2(v.pair(i), splat(K.k2))), splat(1.0f)));
  return fma2(r, splat(K.a2), b2);
}
template <class U>
__device__ __forceinline__ fp2 cap_slope(const U& v, int i, const CapK& K, fp2& E) {
  E = ex2_2(mul2(pair_min(v, i, K), splat(K.k2)));
  return ((kCapBwdFmaPairs >> i) & 1u) ? rcp2_fma_neg(sub2(splat(-1.0f), E)) : rcp2(add2(E, splat(1.0f)));
}

// Online max and sum of one thread's vectors, folded in groups: the group's
// max first, one rescale if it grows.
template <class T, bool CAP>
struct RowSum {
  float m_raw = neg_inf(), m = neg_inf();
  fp2 c2 = 0;   // -centre, or with a cap b2 = (c - m) kk
  fp2 s2 = 0;

  __device__ __forceinline__ void raise(float vmax, const Scale& S) {
    if (vmax > m_raw || (CAP && m == neg_inf())) {
      const float mn = CAP ? cap_zr_rare(vmax, S.K) : vmax;
      s2 = mul2(s2, splat(ex2_rare((m - mn) * S.kk)));
      m_raw = vmax;
      m = mn;
      c2 = splat(CAP ? (S.K.c - mn) * S.kk : -mn);
    }
  }
  // adds the weights of a unit's columns (PARTIAL: of its first `valid`) to `sum`
  template <bool PARTIAL>
  __device__ __forceinline__ void add_to(fp2& sum, const Unit<T>& v, int valid, const Scale& S) const {
    // the unit's own sum first: the total may hold the row's largest weight,
    // next to which single small ones round away
    fp2 unit = 0;
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) {
      fp2 e = ex2_2(CAP ? cap_weight(v, i, S.K, c2) : mul2(add2(v.pair(i), c2), splat(S.kk)));
      if (PARTIAL) {
        float a, b;
        upk(e, a, b);
        e = pk(2 * i < valid ? a : 0.0f, 2 * i + 1 < valid ? b : 0.0f);
      }
      unit = i == 0 ? e : add2(unit, e);
    }
    sum = add2(sum, unit);
  }
  __device__ __forceinline__ MaxSum state() const { return {m, sum2(s2)}; }
};

// --------------------------------------------------------------------------
// A row's run in shared memory.  The copy keeps the run's phase within a
// 16-byte granule, so that all but the ends move in whole granules whatever
// the row's alignment; a unit of columns is then read from one or two granules.
// --------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}

// A unit of columns that starts `shift` elements (uniform over the CTA) behind a
// granule boundary, from the granules there: whole words by SW, known to the
// compiler (with_shift), and for 16-bit types a last half word by a funnel
// shift of `bits`.
template <class T>
struct Granules;
template <class T>
struct Granules16 {
  static constexpr int kPer = 8;   // elements per granule
  __device__ __forceinline__ static int words(int shift) { return shift >> 1; }
  __device__ __forceinline__ static uint32_t bits(int shift) { return (shift & 1) * 16; }
  // load(i): granule i counted from the boundary
  template <class Load>
  __device__ __forceinline__ static void aligned(Unit<T>& r, Load load) {
    const uint4 a = load(0);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  }
  template <int SW, class Load>
  __device__ __forceinline__ static void unit(Unit<T>& r, uint32_t bits, Load load) {
    const uint4 a = load(0), b = load(1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = __funnelshift_r(w[SW + i], w[SW + i + 1], bits);
  }
  // elements j >= valid become -inf
  __device__ __forceinline__ static void clip(Unit<T>& r, int valid) {
    constexpr uint32_t inf = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i >= valid) r.w[i] = inf | (inf << 16);
      else if (2 * i + 1 >= valid) r.w[i] = (r.w[i] & 0xffffu) | (inf << 16);
    }
  }
};
template <>
struct Granules<__nv_bfloat16> : Granules16<__nv_bfloat16> {};
template <>
struct Granules<__half> : Granules16<__half> {};

// Running max over raw vectors: packed words for 16-bit types, unpacked once.
template <class T>
struct RawMax {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  uint32_t w = kBf16 ? kNegInfBf16x2 : kNegInfF16x2;
  __device__ __forceinline__ static uint32_t mx(uint32_t a, uint32_t b) { return kBf16 ? bmax2(a, b) : hmax2(a, b); }
  __device__ __forceinline__ void add(const Unit<T>& x) { w = mx(w, mx(mx(x.w[0], x.w[1]), mx(x.w[2], x.w[3]))); }
  __device__ __forceinline__ float value() const {
    if (kBf16) return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return fmaxf(h2f(w & 0xffffu), h2f(w >> 16));
  }
};
template <>
struct RawMax<float> {
  float m = neg_inf();
  __device__ __forceinline__ void add(const Raw4& x) { m = max3(m, max3(x.v[0], x.v[1], x.v[2]), x.v[3]); }
  __device__ __forceinline__ float value() const { return m; }
};
template <>
struct Granules<float> {
  static constexpr int kPer = 4;
  __device__ __forceinline__ static int words(int shift) { return shift; }
  __device__ __forceinline__ static uint32_t bits(int) { return 0; }
  template <class Load>
  __device__ __forceinline__ static void aligned(Raw4& r, Load load) {
    const uint4 a = load(0);
    r.v[0] = __uint_as_float(a.x); r.v[1] = __uint_as_float(a.y);
    r.v[2] = __uint_as_float(a.z); r.v[3] = __uint_as_float(a.w);
  }
  template <int SW, class Load>
  __device__ __forceinline__ static void unit(Raw4& r, uint32_t, Load load) {
    const uint4 a = load(0);
    uint4 b = make_uint4(0, 0, 0, 0);
    if (SW > 0) b = load(1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = __uint_as_float(w[SW + i]);
  }
  __device__ __forceinline__ static void clip(Raw4& r, int valid) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j >= valid) r.v[j] = neg_inf();
  }
};

// Columns 2i, 2i + 1 of a raw vector from their exact fp32 values.
__device__ __forceinline__ void set_pair(Raw4& r, int i, float a, float b) {
  r.v[2 * i] = a;
  r.v[2 * i + 1] = b;
}
__device__ __forceinline__ void set_pair(Raw8<__nv_bfloat16>& r, int i, float a, float b) {
  r.w[i] = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
}
__device__ __forceinline__ void set_pair(Raw8<__half>& r, int i, float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
}

// f(word shift as a constant, bits) for a shift in elements.
template <class T, class F>
__device__ __forceinline__ void with_shift(int shift, F f) {
  const uint32_t bits = Granules<T>::bits(shift);
  switch (Granules<T>::words(shift)) {
    case 0: f(std::integral_constant<int, 0>{}, bits); break;
    case 1: f(std::integral_constant<int, 1>{}, bits); break;
    case 2: f(std::integral_constant<int, 2>{}, bits); break;
    default: f(std::integral_constant<int, 3>{}, bits); break;
  }
}

template <class T>
__device__ __forceinline__ int phase_of(const T* p) {   // elements behind the last 16-byte boundary
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// Shared memory of a staged run of `cols` columns: the run at any phase, one
// granule in front and two behind (a unit may be read past either end; what
// it holds there is never used).
template <class T>
__host__ __device__ __forceinline__ size_t stage_bytes(int64_t cols) {
  return 16 * (3 + (static_cast<size_t>(cols) + 2 * (16 / sizeof(T))) * sizeof(T) / 16);
}

template <class T, bool ALIGNED>
struct Stage {
  static constexpr int kPer = Granules<T>::kPer;
  uint32_t base;   // shared address of the granule that holds the run's first element
  int phase;       // of the run's first element
  int cols;

  __device__ __forceinline__ Stage(unsigned char* smem, const T* run, int n)
      : base(static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + 16), phase(ALIGNED ? 0 : phase_of(run)), cols(n) {}

  // Starts the copy.  An aligned run: each thread copies the vectors it will
  // sum itself, so that its own wait is enough.
  __device__ __forceinline__ void start(const T* run, unsigned char* smem) const {
    T* own = reinterpret_cast<T*>(smem + 16) + phase;
    if (ALIGNED || phase == 0) {
      static_assert(kCols<T> == kPer, "a unit is a granule");
      const int nvec = (cols + kCols<T> - 1) / kCols<T>;
      for (int v = threadIdx.x; v < nvec; v += kLossThreads) {
        if (kCols<T> * v + kCols<T> <= cols) {
          cp_async16(base + 16u * static_cast<uint32_t>(v), run + kCols<T> * v);
        } else {
          for (int c = kCols<T> * v; c < cols; ++c) own[c] = run[c];
        }
      }
    } else {
      const int head = min(kPer - phase, cols);             // elements before the first boundary
      const int whole = (cols - head) / kPer;               // granules wholly inside the run
      const T* g = run + head;
      const uint32_t dst = base + 16;
      for (int i = threadIdx.x; i < whole; i += kLossThreads) cp_async16(dst + 16 * i, g + i * kPer);
      const int tail = head + whole * kPer;
      if (static_cast<int>(threadIdx.x) < head) own[threadIdx.x] = run[threadIdx.x];
      if (static_cast<int>(threadIdx.x) < cols - tail) own[tail + threadIdx.x] = run[tail + threadIdx.x];
    }
  }
  // the unit from element e on, e + phase a multiple of a granule
  __device__ __forceinline__ void aligned(Unit<T>& r, int e) const {
    const uint32_t g = base + static_cast<uint32_t>((e + phase) * static_cast<int>(sizeof(T)));
    Granules<T>::aligned(r, [&](int i) { return ld_shared16(g + 16 * i); });
  }
  // the same SW words and `bits` behind one (e + phase may be negative by less than a granule)
  template <int SW>
  __device__ __forceinline__ void shifted(Unit<T>& r, int e, uint32_t bits) const {
    const uint32_t g = base + static_cast<uint32_t>(((e + phase) & ~(kPer - 1)) * static_cast<int>(sizeof(T)));
    Granules<T>::template unit<SW>(r, bits, [&](int i) { return ld_shared16(g + 16 * i); });
  }
  __device__ __forceinline__ void unit(Unit<T>& r, int e) const {
    const int shift = ALIGNED ? 0 : (e + phase) & (kPer - 1);
    if (shift == 0) aligned(r, e);
    else with_shift<T>(shift, [&](auto sw, uint32_t bits) { shifted<decltype(sw)::value>(r, e, bits); });
  }
};

// Sum (or max) over a warp, the same bits in every lane: xor 16..1.
template <bool MAX>
__device__ __forceinline__ float warp_all(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  return v;
}

// --------------------------------------------------------------------------
// Targets of a row with k > 1 that lie in this CTA's columns, in shared memory
// and in ascending order of their place j among the row's k: column, j,
// coefficient c_j, logit; and a hash set of the columns, which only tells
// whether one of them occurs twice.
// --------------------------------------------------------------------------
struct Targets {
  int32_t* id;
  int32_t* j;
  float* g;
  float* x;
  int32_t* hash;   // hsize entries
  int hsize;
  int* twice;
};
__host__ __device__ __forceinline__ int target_hash_size(int k) {
  int h = 4;
  while (h < 2 * k) h <<= 1;
  return h;
}
__host__ __device__ __forceinline__ size_t target_smem(int k) {
  return (16 * static_cast<size_t>(k) + 4 * static_cast<size_t>(target_hash_size(k)) + 15) / 16 * 16;
}
__device__ __forceinline__ Targets targets_at(unsigned char* smem, int k, int* twice) {
  Targets t;
  t.id = reinterpret_cast<int32_t*>(smem);
  t.j = t.id + k;
  t.g = reinterpret_cast<float*>(t.j + k);
  t.x = t.g + k;
  t.hash = reinterpret_cast<int32_t*>(t.x + k);
  t.hsize = target_hash_size(k);
  t.twice = twice;
  return t;
}
// All k ids of the row, by `n` threads: t.id (-1 where ignored) and, from
// value(j, valid), t.g.  Behind a barrier of theirs they are collected.
template <class Value>
__device__ __forceinline__ void targets_load(const Targets& t, int at, int n, const int64_t* ids, int k, int64_t V,
                                             int64_t ignore_index, Value value) {
#pragma unroll 2
  for (int j = at; j < k; j += n) {
    const int64_t id = ids[j];
    const bool ok = valid_id(id, V, ignore_index);
    t.id[j] = ok ? static_cast<int32_t>(id) : -1;
    t.g[j] = value(j, ok);
  }
}
// By one warp: keeps the targets in [col_beg, col_end), moved to the front of
// t.id, t.j and t.g, and returns their number; each(g, valid) sees every place
// of the row, in one lane.
template <class Each>
__device__ __forceinline__ int targets_collect(const Targets& t, int k, int64_t col_beg, int64_t col_end, Each each) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 2
  for (int j0 = 0; j0 < k; j0 += 32) {
    const int j = j0 + lane;
    const int32_t id = j < k ? t.id[j] : -1;
    const float g = j < k ? t.g[j] : 0.0f;
    if (j < k) each(g, id >= 0);
    const bool own = id >= col_beg && id < col_end;
    const uint32_t mask = __ballot_sync(0xffffffffu, own);
    __syncwarp();   // the places written below were read before
    if (own) {
      const int at = n + __popc(mask & ((1u << lane) - 1u));
      t.id[at] = id;
      t.j[at] = j;
      t.g[at] = g;
    }
    n += __popc(mask);
  }
  __syncwarp();
  return n;
}
// By one warp: whether one of the n columns occurs twice.  At most n <= k of at
// least 2 k entries are taken: every probe ends at a free or an equal one.
__device__ __forceinline__ void targets_twice(const Targets& t, int n) {
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < t.hsize; i += 32) t.hash[i] = -1;
  __syncwarp();
  bool twice = false;
  for (int i = lane; i < n; i += 32) {
    const int32_t id = t.id[i];
    uint32_t at = (static_cast<uint32_t>(id) * 2654435761u) >> 7;
    for (;; ++at) {
      at &= t.hsize - 1;
      const int32_t old = atomicCAS(&t.hash[at], -1, id);
      if (old == -1) break;
      if (old == id) {
        twice = true;
        break;
      }
    }
  }
  twice = __any_sync(0xffffffffu, twice);
  if (lane == 0) *t.twice = twice;
}

// --------------------------------------------------------------------------
// Gradient of the CTA's columns.
// --------------------------------------------------------------------------
struct GradRow {
  float m, log_s, G;   // G already holds the upstream factor
};

template <class T, bool CAP>
struct GradMap {
  fp2 c2, l2, k2, g2;
  float nm, nl;   // -m; -log2 S, or with a cap the softmax's b2
  __device__ __forceinline__ GradMap(const GradRow& r, const Scale& S) {
    nm = -r.m;
    nl = CAP ? (S.K.c - r.m) * S.kk - r.log_s * kLog2e : -r.log_s * kLog2e;
    c2 = splat(nm);
    k2 = splat(S.kk);
    l2 = splat(nl);
    g2 = splat(-r.G * S.inv_tau * (CAP ? 4.0f : 1.0f));
  }
  __device__ __forceinline__ fp2 pair(const Unit<T>& x, int i, const Scale& S) const {
    if constexpr (CAP) {
      fp2 E;
      const fp2 r = cap_slope(x, i, S.K, E);
      const fp2 p = ex2_2(fma2(r, splat(S.K.a2), l2));
      return mul2(mul2(p, g2), mul2(mul2(E, r), r));
    } else {
      return mul2(ex2_2(fma2(add2(x.pair(i), c2), k2, l2)), g2);
    }
  }
  // (gsum - G q) (dz/dx) / tau at one column
  __device__ __forceinline__ float at(float x, float gsum, const GradRow& r, const Scale& S) const {
    if (CAP) {
      float E;
      const float rr = cap_r_lim(x, S.K, E);
      const float p = ex2(fmaf(rr, S.K.a2, nl));
      return fmaf(-r.G, p, gsum) * S.inv_tau * (4.0f * E * rr * rr);
    }
    const float p = ex2(fmaf(x + nm, S.kk, nl));
    return fmaf(-r.G, p, gsum) * S.inv_tau;
  }
};

template <class T>
__device__ __forceinline__ void fill_vectors(T* dr, int64_t vb, int64_t ve, int64_t V, float value) {
  const bool al = aligned16(dr);
  const fp2 c = splat(value);
  const fp2 o[4] = {c, c, c, c};
  for (int64_t v = vb + threadIdx.x; v < ve; v += kLossThreads) store_vec(dr, v, V, al, o);
}

// 16-byte read-only load that may stay in L1 (a granule that two threads read).
__device__ __forceinline__ uint4 ld_cached16(const void* p) {
  uint4 r;
  asm("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Online max and sum of the thread's units of a run, in groups of U: the group's
// max, a rescale if the max grows, then the group's sum on its own before it
// joins the thread's.  A thread's total may hold the row's largest weight, next
// to which single small weights round away; a group's does so only in the one
// group that holds it.  load(x[U], v): units v, v + kLossThreads, ..., called by
// whole warps none of whose units is the run's last; load_one(x, v): one unit;
// load_last(x, v, valid): the columns behind the last whole unit.
template <int U, class T, bool CAP, class I, class Load, class LoadOne, class LoadLast>
__device__ __forceinline__ void sum_groups(RowSum<T, CAP>& acc, I cols, const Scale& S, Load load, LoadOne load_one,
                                           LoadLast load_last) {
  const I n = cols / kCols<T>;
  I v = threadIdx.x;
  for (; (v | 31) + (U - 1) * kLossThreads + 1 < n; v += U * kLossThreads) {
    Unit<T> x[U];
    load(x, v);
    RawMax<T> mx;
#pragma unroll
    for (int u = 0; u < U; ++u) mx.add(x[u]);
    acc.raise(mx.value(), S);
    fp2 sum = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) acc.template add_to<false>(sum, x[u], kCols<T>, S);
    acc.s2 = add2(acc.s2, sum);
  }
  for (; v < n; v += kLossThreads) {
    Unit<T> x;
    load_one(x, v);
    acc.raise(x.max(), S);
    fp2 sum = 0;
    acc.template add_to<false>(sum, x, kCols<T>, S);
    acc.s2 = add2(acc.s2, sum);
  }
  if (v == n && (cols & (kCols<T> - 1))) {
    Unit<T> x;
    load_last(x, v, static_cast<int>(cols & (kCols<T> - 1)));
    acc.raise(x.max(), S);
    acc.template add_to<true>(acc.s2, x, static_cast<int>(cols & (kCols<T> - 1)), S);
  }
}
// A run in global memory.  ALIGNED: every run starts on a 16-byte boundary; else a
// unit is put together from the two granules that hold it, of which each lane
// loads one and takes the other from its neighbour (element by element at the
// run's ends, whose granules reach outside).  4096 x 151937 bf16: 214 us, against
// 253 when each lane loads both and 193 at 151936 columns.
constexpr int kStreamGroup = 4;
template <bool ALIGNED, class T, bool CAP>
__device__ __forceinline__ void sum_global(RowSum<T, CAP>& acc, const T* run, int64_t cols, const Scale& S) {
  const int shift = ALIGNED ? 0 : phase_of(run);
  auto load_last = [&](Unit<T>& x, int64_t v, int valid) { x.load_scalar(run + kCols<T> * v, valid); };
  if (shift == 0) {
    auto load_one = [&](Unit<T>& x, int64_t v) { x.load(run + kCols<T> * v); };
    sum_groups<kStreamGroup>(
        acc, cols, S,
        [&](Unit<T>* x, int64_t v) {
#pragma unroll
          for (int u = 0; u < kStreamGroup; ++u) load_one(x[u], v + u * kLossThreads);
        },
        load_one, load_last);
  } else if constexpr (!ALIGNED) {
    const int64_t n = cols / kCols<T>;
    with_shift<T>(shift, [&](auto sw, uint32_t bits) {
      constexpr int SW = decltype(sw)::value;
      constexpr int kLast = sizeof(T) == 4 ? -1 : 0;   // 16-bit units may end in the middle of a word
      sum_groups<kStreamGroup>(
          acc, cols, S,
          [&](Unit<T>* x, int64_t v) {
            // a vector's second granule is the next lane's first
            const T* g = run + (kCols<T> * v - shift);
            uint4 first[kStreamGroup], second[kStreamGroup];
#pragma unroll
            for (int u = 0; u < kStreamGroup; ++u)   // (vector 0's first one reaches in front of the run)
              first[u] = ld_stream16(g + kCols<T> * (u * kLossThreads + (u == 0 && v == 0 ? 1 : 0)));
            if ((threadIdx.x & 31) == 31) {
#pragma unroll
              for (int u = 0; u < kStreamGroup; ++u) second[u] = ld_cached16(g + kCols<T> * (u * kLossThreads + 1));
            }
#pragma unroll
            for (int u = 0; u < kStreamGroup; ++u) {
              const bool own = (threadIdx.x & 31) == 31;
              uint4 b = make_uint4(0, 0, 0, 0);
              auto next = [&](uint32_t w, uint32_t mine) {
                const uint32_t o = __shfl_down_sync(0xffffffffu, w, 1);
                return own ? mine : o;
              };
              b.x = next(first[u].x, second[u].x);
              if (SW + kLast > 0) b.y = next(first[u].y, second[u].y);
              if (SW + kLast > 1) b.z = next(first[u].z, second[u].z);
              if (SW + kLast > 2) b.w = next(first[u].w, second[u].w);
              Granules<T>::template unit<SW>(x[u], bits, [&](int i) { return i == 0 ? first[u] : b; });
            }
            if (v == 0) x[0].load_scalar(run, kCols<T>);
          },
          [&](Unit<T>& x, int64_t v) {
            const T* g = run + (kCols<T> * v - shift);
            if (v > 0 && v + 1 < n)
              Granules<T>::template unit<SW>(x, bits, [&](int i) { return ld_cached16(g + i * Granules<T>::kPer); });
            else
              x.load_scalar(run + kCols<T> * v, kCols<T>);
          },
          load_last);
    });
  }
}
// The same over a staged run.  One pass with a running max beats a pass for the
// warp's max and one for the sums (4096 x 151936 bf16 policy 384 us against 396,
// 151937 columns 429 against 458).  Groups of 2 leave more registers than groups
// of 4 (429 against 436 us there; 4096 x 30011 fp16 106 against 109); softcapped
// ones, whose rescale costs two exponentials, are better in fours (2048 x 262144
// bf16 547 us against 559).
template <class T, bool CAP, bool ALIGNED>
__device__ __forceinline__ void sum_staged(RowSum<T, CAP>& acc, const Stage<T, ALIGNED>& run, const Scale& S) {
  constexpr int U = CAP ? 4 : 2;
  auto load_last = [&](Unit<T>& x, int v, int valid) {
    run.unit(x, kCols<T> * v);
    Granules<T>::clip(x, valid);
  };
  auto sum = [&](auto load_one) {
    sum_groups<U>(
        acc, run.cols, S,
        [&](Unit<T>* x, int v) {
#pragma unroll
          for (int u = 0; u < U; ++u) load_one(x[u], v + u * kLossThreads);
        },
        load_one, load_last);
  };
  if (ALIGNED || run.phase == 0)
    sum([&](Unit<T>& x, int v) { run.aligned(x, kCols<T> * v); });
  else
    with_shift<T>(run.phase, [&](auto sw, uint32_t bits) {
      sum([&](Unit<T>& x, int v) { run.template shifted<decltype(sw)::value>(x, kCols<T> * v, bits); });
    });
}

// Writes -G q over a run of `cols` columns read from global memory; the
// one-hot columns follow.  The units of columns are aligned to the gradient
// row's own 16-byte boundaries, so that odd rows are stored in whole vectors
// too, and are read in whole vectors where the logits' row has the same phase
// (contiguous logits), else from the two granules that hold them.  With a cap
// the arithmetic of a column depends on its place within its vector of 8
// columns, so there the units stay on the columns.
template <bool ALIGNED, class T, bool CAP>
__device__ __forceinline__ void grad_global(const T* run, T* dp, int64_t cols, const GradMap<T, CAP>& map,
                                            const Scale& S) {
  constexpr int U = 4;
  constexpr int kPer = Granules<T>::kPer;
  const int po = ALIGNED ? 0 : phase_of(dp), pi = ALIGNED ? 0 : phase_of(run);
  const int lead = CAP ? 0 : po;
  const bool whole = !CAP || po == 0;
  const int64_t units = (cols + lead + kCols<T> - 1) / kCols<T>;
  auto write = [&](int64_t u, const Unit<T>& x) {
    fp2 o[kPairs<T>];
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) o[i] = map.pair(x, i, S);
    store_unit<T>(dp + (kCols<T> * u - lead), o);
  };
  auto edge = [&](int64_t u) {   // element by element
    const int64_t e = kCols<T> * u - lead;
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) {
      Unit<T> x;
      const int64_t c0 = e + 2 * i;
      const bool in0 = c0 >= 0 && c0 < cols, in1 = c0 + 1 >= 0 && c0 + 1 < cols;
      float a = in0 ? load1(run + c0) : 0.0f, b = in1 ? load1(run + c0 + 1) : 0.0f;
      set_pair(x, i, a, b);
      upk(map.pair(x, i, S), a, b);
      if (in0) Out8<T>::store1(dp + c0, a);
      if (in1) Out8<T>::store1(dp + c0 + 1, b);
    }
  };
  int64_t first = 0, end = 0;   // units written in whole vectors
  if (whole && (ALIGNED || pi == lead)) {
    first = lead > 0 ? 1 : 0;
    end = (cols + lead) / kCols<T>;
    int64_t u = first + threadIdx.x;
    for (; u + (U - 1) * kLossThreads < end; u += U * kLossThreads) {
      Unit<T> x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) x[i].load(run + (kCols<T> * (u + i * kLossThreads) - lead));
#pragma unroll
      for (int i = 0; i < U; ++i) write(u + i * kLossThreads, x[i]);
    }
    for (; u < end; u += kLossThreads) {
      Unit<T> x;
      x.load(run + (kCols<T> * u - lead));
      write(u, x);
    }
  } else if constexpr (!ALIGNED) {
   if (whole) {
    // the granules of units [first, end) lie inside the run
    first = 2;
    end = ((cols + lead) / kCols<T>) - 2;
    const int shift = (pi - lead) & (kPer - 1);
    with_shift<T>(shift, [&](auto sw, uint32_t bits) {
#pragma unroll 2
      for (int64_t u = first + threadIdx.x; u < end; u += kLossThreads) {
        Unit<T> x;
        const T* g = run + (kCols<T> * u - lead - shift);
        Granules<T>::template unit<decltype(sw)::value>(x, bits, [&](int i) { return ld_cached16(g + i * kPer); });
        write(u, x);
      }
    });
   }
  }
  if (end < first) end = first;
  for (int64_t u = threadIdx.x; u < min(first, units); u += kLossThreads) edge(u);
  for (int64_t u = end + threadIdx.x; u < units; u += kLossThreads) edge(u);
}

// The same over a staged run.
template <class T, bool CAP, bool ALIGNED>
__device__ __forceinline__ void grad_run(T* dp, const Stage<T, ALIGNED>& run, const GradMap<T, CAP>& map, const Scale& S) {
  const int po = ALIGNED ? 0 : phase_of(dp);
  const int lead = CAP ? 0 : po;
  const bool whole = !CAP || po == 0;   // units are stored in whole vectors
  const int units = (run.cols + lead + kCols<T> - 1) / kCols<T>;
  // units [first, end) lie wholly inside the run
  const int first = whole ? (lead > 0 ? 1 : 0) : units;
  const int end = whole ? (run.cols + lead) / kCols<T> : 0;
  auto write = [&](int u, const Unit<T>& x) {
    fp2 o[kPairs<T>];
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) o[i] = map.pair(x, i, S);
    store_unit<T>(dp + (kCols<T> * u - lead), o);
  };
  if (ALIGNED || run.phase == lead) {
#pragma unroll 2
    for (int u = first + threadIdx.x; u < end; u += kLossThreads) {
      Unit<T> x;
      run.aligned(x, kCols<T> * u - lead);
      write(u, x);
    }
  } else {
    with_shift<T>((run.phase - lead) & (Granules<T>::kPer - 1), [&](auto sw, uint32_t bits) {
      for (int u = first + threadIdx.x; u < end; u += kLossThreads) {
        Unit<T> x;
        run.template shifted<decltype(sw)::value>(x, kCols<T> * u - lead, bits);
        write(u, x);
      }
    });
  }
  // the units that reach over an end (all of them where none is whole)
  auto edge = [&](int u) {
    const int e = kCols<T> * u - lead;
    Unit<T> x;
    run.unit(x, e);
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) {
      float a, b;
      upk(map.pair(x, i, S), a, b);
      if (e + 2 * i >= 0 && e + 2 * i < run.cols) Out8<T>::store1(dp + e + 2 * i, a);
      if (e + 2 * i + 1 >= 0 && e + 2 * i + 1 < run.cols) Out8<T>::store1(dp + e + 2 * i + 1, b);
    }
  };
  const int from = whole ? max(first, end) : 0;
  if (whole && static_cast<int>(threadIdx.x) < first) edge(threadIdx.x);
  for (int u = from + threadIdx.x; u < units; u += kLossThreads) edge(u);
}

// Rewrites the one-hot columns of the CTA's n targets, after a barrier behind
// the gradient's vectors.  Duplicate columns: the first of them writes the sum
// of all their coefficients in ascending j.
template <class T, bool CAP>
__device__ __forceinline__ void grad_targets(T* dr, const Targets& t, int n, const GradMap<T, CAP>& map,
                                             const GradRow& r, const Scale& S) {
  const bool twice = *t.twice != 0;
  for (int i = threadIdx.x; i < n; i += kLossThreads) {
    const int32_t id = t.id[i];
    float gs = t.g[i];
    if (twice) {
      bool first = true;
      for (int o = 0; o < i; ++o) first = first && t.id[o] != id;
      if (!first) continue;
      for (int o = i + 1; o < n; ++o) {
        if (t.id[o] == id) gs += t.g[o];
      }
    }
    Out8<T>::store1(dr + id, map.at(t.x[i], gs, r, S));
  }
}

// --------------------------------------------------------------------------
// The losses.
// --------------------------------------------------------------------------

// Clipped policy loss of one token.  A: advantage, r = exp(logp - old):
//   pg = -min(r A, clip(r, lo, hi) A), for A < 0 at most -dual A (dual > 0),
//   kl = exp(ref - logp) - (ref - logp) - 1,
//   L = pg + beta kl,
// and dL/dlogp.  A token whose clipped term is the smaller one has no pg
// gradient; at a border both terms agree and the gradient passes.  Comparisons
// are written so that a NaN ratio or advantage makes the loss and the gradient NaN.
struct Token {
  float old, adv, ref, w;
};
__device__ __forceinline__ float policy_token(float logp, const Token& t, float lo, float hi, float dual, bool kl,
                                              float beta, float* loss) {
  const float adv = t.adv;
  const float r = expf(logp - t.old);
  const float rc = r < lo ? lo : (r > hi ? hi : r);
  // a ratio beyond fp32 (log r > 88) of a finite old_logp times 0 is 0
  const float s1 = adv == 0.0f && r == pos_inf() && t.old > neg_inf() ? 0.0f : r * adv, s2 = rc * adv;
  float gain = s2 < s1 ? s2 : s1;
  float d = (rc == r || !(s1 >= s2)) ? -s1 : 0.0f;
  if (dual > 0.0f && adv < 0.0f) {
    const float least = dual * adv;
    if (gain <= least) {
      gain = least;
      d = 0.0f;
    }
  }
  float L = -gain;
  if (kl) {
    const float e = t.ref - logp, x = expm1f(e);
    L = fmaf(beta, x - e, L);
    d = fmaf(-beta, x, d);
  }
  *loss = L;
  return d;
}

__device__ __forceinline__ float load_teacher(const void* p, int dt, int64_t i) {
  if (dt == VLS_F32) return __ldg(static_cast<const float*>(p) + i);
  if (dt == VLS_BF16) return load1(static_cast<const __nv_bfloat16*>(p) + i);
  return load1(static_cast<const __half*>(p) + i);
}

// A barrier of the kLossThreads threads that sweep the row.
__device__ __forceinline__ void sweep_sync() { asm volatile("bar.sync 2, %0;" ::"n"(kLossThreads) : "memory"); }

// What a distillation row needs beside the sums over the vocabulary, none of it
// depending on them (so it overlaps the loads).  Each CTA of the row's cluster
// takes the targets of its own columns: with t_j the teacher's logits, base and
// z0 the largest t_j and z_j among them, e_j = exp((t_j - base) / tau),
//   P = sum e_j,   B = sum e_j ((t_j - base) - (z_j - z0)) / tau.
// With b the largest base of the row's CTAs, s = b / tau - teacher_lse (0 without
// it), f = exp((base - b) / tau + s) and Z the sum of f P over the CTAs (1 with
// teacher_lse), the teacher's probabilities are p_j = f e_j / Z and the row's loss
// is the sum over CTAs of
//   f / Z (B + P ((base - b) / tau + s - log Z + (m - z0) / tau + log S)).
// Logits are subtracted before they are scaled: a difference of two near ones is
// exact, while t_j / tau is rounded at the size of t_j (at offset -8192 and tau =
// 0.7 that alone moved p_j by 8e-4).  s, a difference of two large numbers, takes
// 1 / tau in two floats.
struct DistillPart {
  float P, B, z0, base;   // B times tau
};
// Three floats: with five, 16 bytes more of static shared memory, only 4 CTAs of
// 43 KB and 64 targets fit an SM instead of 5 (4096 x 151936 bf16: 424 us, 405).
struct DistillRow {
  float b, shift, scale;   // c_j = scale 2^((t_j - b) kk + shift), kk = log2(e) / tau
  __device__ __forceinline__ float weight(float t, float kk) const { return ex2(fmaf(t - b, kk, shift)); }
};

// One entry's share of P and B.
template <bool CAP>
__device__ __forceinline__ void part_add(float t, float x, float bc, float z0, const Scale& S, float& P, float& B) {
  const float d = t - bc, e = ex2(d * S.kk);
  const float z = CAP ? cap_zr(x, S.K) : x;
  P += e;
  if (e != 0.0f) B += e * (d - (z - z0));
}
// Sums P and B over the warp (xor 16 exchanges one for the other, then 8..1)
// and writes the part.
__device__ __forceinline__ void part_write(float P, float B, float base, float z0, DistillPart* out) {
  const int lane = threadIdx.x & 31;
  const bool high = (lane & 16) != 0;
  float v = high ? B : P;
  v += __shfl_xor_sync(0xffffffffu, high ? P : B, 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (lane == 0) {
    out->P = v;
    out->z0 = z0;
    out->base = base;
  }
  if (lane == 16) out->B = v;
}

// Rows with more targets have kernels of their own, which leaves these their
// registers (4096 x 151936 bf16 k = 64: 404 us, 470 in one kernel).
constexpr int kFewTargets = 64;
// By one warp; returns the number of this CTA's targets.  A single warp beside
// 40 busy ones takes some 20 cycles an instruction, so this one's instructions
// are what a row waits for; the entries stay in registers, two a lane.
template <class T, bool CAP>
__device__ __forceinline__ int distill_few(const LossArgs& a, int64_t row, bool first, const T* xr, int64_t col_beg,
                                           int64_t col_end, const Targets& t, const Scale& S, DistillPart* out) {
  const int lane = threadIdx.x & 31, k = a.k;
  const int64_t at = row * k;
  int32_t id[2];
  float lt[2], x[2], base = neg_inf(), zm = neg_inf();
  uint32_t own[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    const int64_t id64 = j < k ? a.ids[at + j] : -1;
    lt[i] = j < k ? load_teacher(a.teacher, a.teacher_dt, at + j) : 0.0f;
    const bool ok = valid_id(id64, a.vocab, a.ignore_index);
    if (first && !ok && j < k) a.coef[at + j] = 0.0f;
    id[i] = static_cast<int32_t>(id64);
    own[i] = __ballot_sync(0xffffffffu, ok && id64 >= col_beg && id64 < col_end);
    const bool mine = (own[i] >> lane) & 1u;
    x[i] = mine ? load1(xr + id[i]) : neg_inf();
    if (mine) base = fmaxf(base, lt[i]);
  }
  base = warp_max(base);
  const float bc = centre(base);
  int n = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if ((own[i] >> lane) & 1u) {
      const int to = n + __popc(own[i] & ((1u << lane) - 1u));
      t.id[to] = id[i];
      t.j[to] = lane + 32 * i;
      t.g[to] = lt[i];
      t.x[to] = x[i];
      zm = fmaxf(zm, CAP ? cap_zr(x[i], S.K) : x[i]);
    }
    n += __popc(own[i]);
  }
  const float z0 = centre(warp_max(zm));
  float P = 0.0f, B = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if ((own[i] >> lane) & 1u) part_add<CAP>(lt[i], x[i], bc, z0, S, P, B);
  }
  part_write(P, B, base, z0, out);
  __syncwarp();
  return n;
}
// More than 64: the row's other eight warps find this CTA's targets and load
// their logits, each thread up to 4 of the k; the ninth forms the part (4096 x
// 151936 bf16 k = 1024 919 us, 1101 when the ninth did all of it).
static_assert(VLS_MAX_TOPK <= 4 * kLossThreads, "a thread takes up to 4 targets");
constexpr int kTargetWords = VLS_MAX_TOPK / 32;
template <class T>
__device__ __forceinline__ void distill_collect(const LossArgs& a, int64_t row, bool first, const T* xr, int64_t col_beg,
                                                int64_t col_end, const Targets& t, uint32_t* masks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t at = row * a.k;
  int32_t id[4];
  float lt[4];
  uint32_t own[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    own[c] = 0;
    if (c * kLossThreads >= a.k) continue;
    const int j = c * kLossThreads + threadIdx.x;
    const int64_t id64 = j < a.k ? a.ids[at + j] : -1;
    lt[c] = j < a.k ? load_teacher(a.teacher, a.teacher_dt, at + j) : 0.0f;
    const bool ok = valid_id(id64, a.vocab, a.ignore_index);
    if (first && !ok && j < a.k) a.coef[at + j] = 0.0f;
    id[c] = static_cast<int32_t>(id64);
    own[c] = __ballot_sync(0xffffffffu, ok && id64 >= col_beg && id64 < col_end);
    if (lane == 0) masks[c * kLossWarps + warp] = own[c];
  }
  sweep_sync();
  int before = 0, word = 0;   // targets in the words before this one's
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    if (c * kLossThreads >= a.k) continue;
    for (; word < c * kLossWarps + warp; ++word) before += __popc(masks[word]);
    if ((own[c] >> lane) & 1u) {
      const int to = before + __popc(own[c] & ((1u << lane) - 1u));
      t.id[to] = id[c];
      t.j[to] = c * kLossThreads + threadIdx.x;
      t.g[to] = lt[c];
      t.x[to] = load1(xr + id[c]);
    }
  }
}
template <bool CAP>
__device__ __forceinline__ int distill_many(int k, const Targets& t, const Scale& S, const uint32_t* masks,
                                            DistillPart* out) {
  const int lane = threadIdx.x & 31;
  // a chunk of kLossThreads targets writes all its words
  const bool written = lane < (k + kLossThreads - 1) / kLossThreads * kLossWarps;
  const int n = __reduce_add_sync(0xffffffffu, written ? __popc(masks[lane]) : 0);
  float base = neg_inf(), zm = neg_inf();
#pragma unroll 2
  for (int i = lane; i < n; i += 32) {
    base = fmaxf(base, t.g[i]);
    zm = fmaxf(zm, CAP ? cap_zr(t.x[i], S.K) : t.x[i]);
  }
  base = warp_max(base);
  const float z0 = centre(warp_max(zm)), bc = centre(base);
  float P = 0.0f, B = 0.0f;
  for (int i = lane; i < n; i += 32) part_add<CAP>(t.g[i], t.x[i], bc, z0, S, P, B);
  part_write(P, B, base, z0, out);
  return n;
}

// The row's loss, G and coefficients from its C CTAs' parts; warp 0.
__device__ __forceinline__ float distill_finish(const DistillPart* parts, int C, float M, const LogSum& ls,
                                                const Scale& S, float inv_tau_lo, bool known, float lse, float w,
                                                DistillRow* r, float* G) {
  const int lane = threadIdx.x & 31;
  const DistillPart d = lane < C ? parts[lane] : DistillPart{0.0f, 0.0f, 0.0f, neg_inf()};
  const float top = warp_all<true>(d.base), b = centre(top), base = centre(d.base);
  const float shift = known ? fmaf(b, S.inv_tau, -lse) + b * inv_tau_lo : 0.0f;
  *r = DistillRow{b, shift * kLog2e, 0.0f};
  // a CTA without targets, or all of whose e_j are 0, takes no part
  const float f = d.P == 0.0f ? 0.0f : r->weight(base, S.kk);
  float Z = 1.0f, P = f * d.P;
#pragma unroll
  for (int off = kLossMaxCluster / 2; off > 0; off >>= 1) P += __shfl_xor_sync(0xffffffffu, P, off);
  if (!known) Z = P;
  const float inv = 1.0f / Z;
  r->scale = -w * inv;
  // log S - log Z from their parts: two numbers of like size that nearly cancel
  const LogSum lz = known ? LogSum{0.0f, 0.0f} : log_sum(Z);
  const float logs = fmaf(ls.e - lz.e, kLn2, ls.lf - lz.lf) + shift;
  float L = f != 0.0f ? f * fmaf(S.inv_tau, d.B, d.P * fmaf((base - b) + (M - d.z0), S.inv_tau, logs)) : 0.0f;
#pragma unroll
  for (int off = kLossMaxCluster / 2; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  *G = -w * (P * inv);
  return (known ? lse : top) == neg_inf() ? qnan() : L * inv;
}

// Whether a row has a valid id; most often its first one says so.
__device__ __forceinline__ bool any_target(const LossArgs& a, int64_t row) {
  const int64_t* ids = a.ids + row * a.k;
  if (valid_id(ids[0], a.vocab, a.ignore_index)) return true;
  if (a.k == 1) return false;
  int any = 0;
  for (int j = threadIdx.x; j < a.k; j += blockDim.x) any |= valid_id(ids[j], a.vocab, a.ignore_index);
  return __syncthreads_or(any) != 0;
}

// --------------------------------------------------------------------------
// The row kernel: statistics, loss and (a.dx) gradient of one row.
// --------------------------------------------------------------------------
// A row's loss outputs and the constants of its gradient; one thread of each
// CTA, the same in all of them (`first`: the one that writes).
template <int LOSS, bool CAP>
__device__ __forceinline__ GradRow finish_row(const LossArgs& a, int64_t row, bool first, const MaxSum& st,
                                              const LogSum& ls, float xt, const Token& tok, float dist_loss,
                                              float dist_G, const Scale& S) {
  float loss = dist_loss, G = dist_G, logp = 0.0f;
  const float log_s = ls.value();
  if constexpr (LOSS != kLossDistill) {
    const float d = CAP ? fmaf(cap_r(xt, S.K), S.K.a2, (S.K.c - st.m) * S.kk) * kLn2
                        : (xt - st.m) * S.inv_tau;
    logp = ls.sub_from(d);
    if constexpr (LOSS == kLossPolicy)
      G = tok.w * policy_token(logp, tok, a.clip_lo, a.clip_hi, a.dual_clip, a.ref_logp != nullptr, a.kl_coef, &loss);
  }
  if (first) {
    a.stats[row] = vls_rowstat{st.m, log_s};
    if (a.row_loss != nullptr) a.row_loss[row] = loss;
    if (LOSS != kLossDistill) {
      a.logp[row] = logp;
      if (a.coef != nullptr) a.coef[row] = G;
    }
  }
  return GradRow{st.m, log_s, G};
}

__device__ __forceinline__ Token load_token(const LossArgs& a, int64_t row) {
  Token t{a.old_logp[row], a.adv[row], 0.0f, 1.0f};
  if (a.ref_logp != nullptr) t.ref = a.ref_logp[row];
  if (a.weights != nullptr) t.w = a.weights[row];
  return t;
}

// Outputs of a row without a target (kLossThreads threads of each of its CTAs).
template <class T>
__device__ __forceinline__ void empty_row(const LossArgs& a, int64_t row, bool first, T* dr, int64_t vb, int64_t ve) {
  if (a.dx != nullptr) fill_vectors(dr, vb, ve, a.vocab, 0.0f);
  if (!first) return;
  for (int j = threadIdx.x; j < a.k; j += kLossThreads) {
    if (a.coef != nullptr) a.coef[row * a.k + j] = 0.0f;
    if (a.logp != nullptr) a.logp[row * a.k + j] = 0.0f;
  }
  if (threadIdx.x == 0) {
    if (a.row_loss != nullptr) a.row_loss[row] = 0.0f;
    a.stats[row] = vls_rowstat{0.0f, 0.0f};
  }
}

// A distillation row has a ninth warp, which forms the targets' part while the
// other eight copy and sum the row.
template <int LOSS>
constexpr int row_threads() { return kLossThreads + (LOSS == kLossDistill ? 32 : 0); }

// Starts pulling bytes (a multiple of 16) at p (16-byte aligned) into L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// Starts the way to L2 of a run by one warp (whole granules of it).
template <class T>
__device__ __forceinline__ void prefetch_run(const T* run, int64_t cols) {
  const uintptr_t beg = (reinterpret_cast<uintptr_t>(run) + 15) & ~static_cast<uintptr_t>(15);
  const uintptr_t end = reinterpret_cast<uintptr_t>(run + cols) & ~static_cast<uintptr_t>(15);
  for (uintptr_t p = beg + (threadIdx.x & 31) * 8192u; p < end; p += 32u * 8192u)
    prefetch_l2_bulk(reinterpret_cast<const void*>(p), static_cast<uint32_t>(end - p < 8192u ? end - p : 8192u));
}

// CTAs an SM that the registers must leave room for.  Staged rows: as many as
// their runs leave room for in shared memory, but a distillation row at odd
// addresses, whose ninth warp takes it over the registers (4096 x 30011 fp16: 110
// us at 4, 115 at 5).  Streamed log-probabilities with their pair launch: 4096 x
// 151936 bf16 193 us at 6, 194 at 5, 196 at 8; at odd addresses 4096 x 30011 fp16
// 64 us at 5, 68 at 6, 66 at 4.
template <class T, int LOSS, bool CAP, bool ALIGNED>
constexpr int loss_min_blocks() {
  if (sizeof(T) == 4) return 4;
  if (LOSS == kLossDistill) return ALIGNED ? 5 : 4;
  return LOSS == kLossLogp && !CAP && ALIGNED ? 6 : 5;
}

// STAGED: the run is copied into shared memory once, and the sums and the
// gradient are taken from there; otherwise (log-probabilities alone, and rows too
// long for the shared memory of a cluster) the sums, and then the gradient, read
// the row from global memory.
//
// What bounds it, and times with the gradient (bytes: one read, one write):
//  - aligned 16-bit rows, memory: 4096 x 151936 bf16 policy 386 us (6.5 TB/s),
//    distillation k = 64 405 us, 18750 x 32000 bf16 policy 363 us (6.6 TB/s).
//    A statistics kernel and a gradient kernel in turn read the logits twice: 193
//    + 368 us at the first of these;
//  - fp32, memory, with 3 or 4 CTAs an SM: 2048 x 151936 policy 384 us (6.5 TB/s),
//    1024 x 262144 406 us (5.3 TB/s);
//  - rows at odd addresses, memory and issue: a unit of columns is put together
//    from two granules: 4096 x 151937 bf16 policy 431 us (5.8 TB/s);
//  - 16-bit rows of 44 to 64 KB, latency: 3 CTAs of 8 warps fill an SM's shared
//    memory, and neither memory (63%) nor issue (56%) is at its limit: 4096 x 30011
//    fp16 107 us (4.6 TB/s), 30008 columns, which are aligned, 100 us;
//  - softcapped rows, latency and issue: two exponentials and a reciprocal a column
//    and sweep in dependent steps, the special-function unit 62% and the issue slots
//    74% busy; 2048 x 262144 bf16 547 us (3.9 TB/s), 326 of them without the
//    gradient;
//  - few rows, latency (a row's chain copy, sum, cluster exchange, store): 8 x
//    32000 bf16 7 us, 16 x 151936 k = 20 distillation 9 us, the loss's sum included.
// One cluster a row and launch beats clusters that stay and refill their shared
// memory row by row (4096 x 151936: 431 us at the best run length, when this one
// took 397: their loads wait for the slowest CTA of the cluster).
template <class T, int LOSS, bool CAP, bool STAGED, bool ALIGNED, bool MANY>
__global__ void __launch_bounds__(row_threads<LOSS>(), (loss_min_blocks<T, LOSS, CAP, ALIGNED>()))
    row_loss_kernel(const LossArgs a) {
  constexpr bool HELP = LOSS == kLossDistill;
  __shared__ MaxSum warp_part[kLossWarps];
  __shared__ MaxSum cta_part[kLossMaxCluster];
  __shared__ DistillPart dist_part[kLossMaxCluster], s_part;
  __shared__ DistillRow s_dist;
  __shared__ uint32_t s_masks[MANY ? kTargetWords : 1];
  __shared__ GradRow s_grad;
  __shared__ int s_twice, s_n;
  extern __shared__ __align__(16) unsigned char dyn[];

  dependents_may_launch();
  const int C = a.cluster;
  const uint32_t row32 = blockIdx.x / static_cast<uint32_t>(C);
  const int64_t row = row32;
  const int q = static_cast<int>(blockIdx.x - row32 * static_cast<uint32_t>(C));
  const int64_t V = a.vocab;
  const int64_t nvec = (V + 7) >> 3;
  const int64_t vb = static_cast<int64_t>(q) * a.vec_per_cta;
  const int64_t ve = min(vb + a.vec_per_cta, nvec);
  const int64_t col_beg = 8 * vb, col_end = min(8 * ve, V);
  const T* xr = row_ptr<T>(a.x, a.rx, row);
  T* dr = static_cast<T*>(a.dx) + row * V;
  const Scale S = make_scale(a.cap, a.inv_tau);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool helper = HELP && warp >= kLossWarps;
  const int64_t next = row + a.ahead;

  // ---- a row without a target is not read ----
  int64_t id = -1;
  bool any;
  if constexpr (HELP) {
    any = any_target(a, row);
  } else {
    id = a.ids[row];
    any = valid_id(id, V, a.ignore_index);
  }
  if (!any) {
    if (!helper) empty_row(a, row, q == 0, dr, vb, ve);
    return;   // the same decision in every CTA of the cluster
  }
  if (C > 1) cluster_arrive_relaxed();

  unsigned char* const staged = dyn + (HELP ? target_smem(a.k) : 0);
  const Stage<T, ALIGNED> stage(staged, xr + col_beg, static_cast<int>(STAGED ? col_end - col_beg : 0));
  const Targets t = targets_at(dyn, a.k, &s_twice);
  float xt = 0.0f;
  Token tok{0.0f, 0.0f, 0.0f, 1.0f};
  MaxSum st{neg_inf(), 0.0f};
  int helped = 0;
  constexpr bool few = !MANY;

  if (helper) {
    // As below for the row, and twice as far ahead its targets: a row's ids
    // decide whether it is copied, and each row's lie in lines of their own.
    int64_t next_id = -1;
    if (STAGED && a.ahead > 0) {
      if (next < a.rows) next_id = a.ids[next * a.k];
      if (next + a.ahead < a.rows) {
        const int64_t at = (next + a.ahead) * a.k;
        for (int j = lane * 16; j < a.k; j += 512) prefetch_l2(a.ids + at + j);
        const int esize = a.teacher_dt == VLS_F32 ? 4 : 2;
        for (int j = lane * 128; j < a.k * esize; j += 4096)
          prefetch_l2(static_cast<const char*>(a.teacher) + at * esize + j);
      }
    }
    if constexpr (few) {
      helped = distill_few<T, CAP>(a, row, q == 0, xr, col_beg, col_end, t, S, &s_part);
    } else {
      asm volatile("bar.sync 3, %0;" ::"n"(kLossThreads + 32) : "memory");
      helped = distill_many<CAP>(a.k, t, S, s_masks, &s_part);
    }
    if (lane == 0) s_n = helped;
    if (valid_id(next_id, V, a.ignore_index))
      prefetch_run(row_ptr<T>(a.x, a.rx, next) + col_beg, col_end - col_beg);
  } else {
    if constexpr (STAGED) stage.start(xr + col_beg, staged);
    if (HELP && warp == 0) {   // read early: their latency overlaps the row's
      if (a.weights != nullptr) tok.w = a.weights[row];
      if (a.teacher_lse != nullptr) tok.ref = a.teacher_lse[row];
    }
    if constexpr (HELP && !few) {
      distill_collect(a, row, q == 0, xr, col_beg, col_end, t, s_masks);
      asm volatile("bar.arrive 3, %0;" ::"n"(kLossThreads + 32) : "memory");
    }
    if constexpr (!HELP) {
      xt = load1(xr + id);
      if (LOSS == kLossPolicy && threadIdx.x == 0) tok = load_token(a, row);   // their latency overlaps the row's
    }
    // The row that will take this one's place starts its way to L2, so that its
    // copy waits for L2 instead of DRAM.
    if (STAGED && !HELP && a.ahead > 0 && warp == kLossWarps - 1 && next < a.rows &&
        valid_id(a.ids[next * a.k], V, a.ignore_index))
      prefetch_run(row_ptr<T>(a.x, a.rx, next) + col_beg, col_end - col_beg);

    // ---- statistics ----
    RowSum<T, CAP> acc;
    if constexpr (STAGED) {
      cp_async_wait();
      if (!ALIGNED && stage.phase != 0) sweep_sync();
      sum_staged(acc, stage, S);
    } else {
      sum_global<ALIGNED>(acc, xr + col_beg, col_end - col_beg, S);
    }
    // ---- combine: lanes, warps, cluster ranks; warp 0 ends with the row's ----
    st = merge_lanes<32>(acc.state(), 32, S.kk);
    if (lane == 0) warp_part[warp] = st;
  }
  __syncthreads();
  if (warp == 0) {
    st = merge_lanes<kLossWarps>(warp_part[lane & (kLossWarps - 1)], kLossWarps, S.kk);
    st.s = __shfl_sync(0xffffffffu, st.s, 0);   // up to 16 lanes hand it on
  }
  if (C > 1) {
    cluster_wait();   // every CTA of the cluster is resident: its shared memory may be written
    if (threadIdx.x < C) {
      cg::this_cluster().map_shared_rank(cta_part, threadIdx.x)[q] = st;
      if (HELP) cg::this_cluster().map_shared_rank(dist_part, threadIdx.x)[q] = s_part;
    }
    cluster_arrive();
  }
  if (helper) {   // while the others meet
    targets_twice(t, helped);
    __syncwarp();
  }
  if (C > 1) cluster_wait();
  // ---- loss: the same in every CTA of the cluster ----
  if (warp == 0) {
    if (C > 1) st = merge_lanes<kLossMaxCluster>(cta_part[lane & (kLossMaxCluster - 1)], C, S.kk);
    const LogSum ls = log_sum(st.m == neg_inf() ? qnan() : st.s);   // all -inf: no distribution
    float dl = 0.0f, G = 0.0f;
    DistillRow dist;
    if constexpr (HELP)
      dl = distill_finish(C > 1 ? dist_part : &s_part, C, st.m, ls, S, a.inv_tau_lo,
                          a.teacher_lse != nullptr, tok.ref, tok.w, &dist, &G);
    if (lane == 0) {
      s_grad = finish_row<LOSS, CAP>(a, row, q == 0, st, ls, xt, tok, dl, G, S);
      if (HELP) s_dist = dist;
    }
  }
  if (LOSS == kLossLogp || (!HELP && a.dx == nullptr)) return;
  __syncthreads();
  if (helper) return;
  const GradRow gr = s_grad;
  if constexpr (HELP) {
    for (int i = threadIdx.x; i < s_n; i += kLossThreads) {
      const float c = s_dist.scale * s_dist.weight(t.g[i], S.kk);
      t.g[i] = c;
      a.coef[row * a.k + t.j[i]] = c;
    }
    if (a.dx == nullptr) return;
  }

  // ---- gradient ----
  if (gr.m == neg_inf()) {
    fill_vectors(dr, vb, ve, V, qnan());
    return;
  }
  const GradMap<T, CAP> map(gr, S);
  if constexpr (STAGED)
    grad_run<T, CAP>(dr + col_beg, stage, map, S);
  else
    grad_global<ALIGNED, T, CAP>(xr + col_beg, dr + col_beg, col_end - col_beg, map, S);
  if constexpr (HELP) {
    sweep_sync();
    grad_targets<T, CAP>(dr, t, s_n, map, gr, S);
  } else {
    if (id >= col_beg && id < col_end) {
      sweep_sync();
      if (threadIdx.x == 0) Out8<T>::store1(dr + id, map.at(xt, gr.G, gr, S));
    }
  }
}

// --------------------------------------------------------------------------
// Sums kept as two floats, hi + lo (about 46 bits): each addition's rounding
// error is computed exactly and carried in lo.  (The GPU's fp64 rate made the
// same sums in fp64 the longest part of their kernels: 56 us at 4096 rows.)
// --------------------------------------------------------------------------
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum2& o) {
    add(o.hi);
    lo += o.lo;
  }
  // an infinite or NaN hi is the sum; lo then holds the NaN of inf - inf
  __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
  __device__ __forceinline__ Sum2 shfl_xor(int m) const {
    return {__shfl_xor_sync(0xffffffffu, hi, m), __shfl_xor_sync(0xffffffffu, lo, m)};
  }
};

// Sum over a CTA (whole warps, at most 32) in a fixed order, in warp 0's lanes.
// buf: 32 entries.
__device__ __forceinline__ Sum2 cta_sum(Sum2 s, Sum2* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const Sum2 o = s.shfl_xor(off);
    s.add(o);
  }
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = threadIdx.x < (blockDim.x >> 5) ? buf[threadIdx.x] : Sum2{0.0f, 0.0f};
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const Sum2 o = s.shfl_xor(off);
      s.add(o);
    }
  }
  return s;
}

// *out = sum_i w_i v_i (w null: 1), products and sum in two floats; one CTA.
static __device__ __noinline__ void weighted_sum(const float* v, const float* w, int64_t n, float* out) {
  __shared__ Sum2 buf[32];
  Sum2 s{0.0f, 0.0f};
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const float x = v[i], y = w != nullptr ? w[i] : 1.0f;
    const float p = x * y;
    s.add(Sum2{p, isfinite(p) ? fmaf(x, y, -p) : 0.0f});
  }
  s = cta_sum(s, buf);
  if (threadIdx.x == 0) *out = s.value();
}

// --------------------------------------------------------------------------
// The gradient alone, from saved statistics and coefficients, times *up: a map
// (one read, one write), bound by memory: 4096 x 151936 bf16 368 us (6.8 TB/s),
// 4096 x 30011 fp16 88 us (5.6 TB/s).  Rows are cut into pieces (chunks) where
// there are few of them; 5 CTAs an SM with 4 vectors of 16 bytes in flight a thread.
// --------------------------------------------------------------------------
template <class T, bool CAP, bool ALIGNED, bool TOPK>
__global__ void __launch_bounds__(kLossThreads, 5) loss_grad_kernel(const LossGradArgs a) {
  __shared__ float s_G;
  __shared__ int s_twice, s_n, s_any;
  extern __shared__ __align__(16) unsigned char dyn[];
  wait_for_previous();
  if (!TOPK && blockIdx.x == static_cast<uint32_t>(a.rows * a.chunks)) {   // a CTA of its own, where it is asked for
    weighted_sum(a.sum_v, a.sum_w, a.sum_n, a.sum_out);
    return;
  }
  const float up = a.up != nullptr ? *a.up : 1.0f;
  if (a.skip_one && up == 1.0f) return;
  // rows from the last to the first: the launch before it read them in order,
  // so the last ones may still be in L2
  const uint32_t row32 = blockIdx.x / static_cast<uint32_t>(a.chunks);
  const int64_t row = a.rows - 1 - row32;
  const int q = static_cast<int>(blockIdx.x - row32 * static_cast<uint32_t>(a.chunks));
  const int64_t V = a.vocab;
  const int64_t nvec = (V + 7) >> 3;
  const int64_t vb = static_cast<int64_t>(q) * a.vec_per_cta;
  const int64_t ve = min(vb + a.vec_per_cta, nvec);
  const int64_t col_beg = 8 * vb, col_end = min(8 * ve, V);
  const T* xr = row_ptr<T>(a.x, a.rx, row);
  T* dr = static_cast<T*>(a.dx) + row * V;
  const Scale S = make_scale(a.cap, a.inv_tau);

  const vls_rowstat st = a.stats[row];
  GradRow gr{st.m, st.log_s, 0.0f};
  int64_t id = -1;
  bool any;
  const Targets t = targets_at(dyn, a.k, &s_twice);
  if constexpr (!TOPK) {
    id = a.ids[row];
    any = valid_id(id, V, a.ignore_index);
    if (any) {
      const float c = a.coef[row];
      // A row that takes no part in its loss has statistics 0.  A row's own may be
      // 0 as well, but then its logits are finite or -inf, and a coefficient of 0
      // makes its gradient 0 all the same.
      any = c != 0.0f || st.m != 0.0f || st.log_s != 0.0f;
      gr.G = c * up;
    }
  } else {
    targets_load(t, threadIdx.x, kLossThreads, a.ids + row * a.k, a.k, V, a.ignore_index,
                 [&](int j, bool ok) { return ok ? a.coef[row * a.k + j] : 0.0f; });
    __syncthreads();
    if (threadIdx.x < 32) {
      float G = 0.0f;
      bool ok_any = false;
      const int n = targets_collect(t, a.k, col_beg, col_end, [&](float g, bool ok) {
        G += g;
        ok_any |= ok;
      });
      G = warp_all<false>(G);
      for (int i = threadIdx.x; i < n; i += 32) {
        t.x[i] = load1(xr + t.id[i]);
        t.g[i] *= up;
      }
      targets_twice(t, n);
      ok_any = __any_sync(0xffffffffu, ok_any);
      if (threadIdx.x == 0) {
        s_G = G;
        s_n = n;
        s_any = ok_any;
      }
    }
    __syncthreads();
    any = s_any;
    gr.G = s_G * up;
  }
  if (!any || st.m == neg_inf()) {
    fill_vectors(dr, vb, ve, V, any ? qnan() : 0.0f);
    return;
  }
  const GradMap<T, CAP> map(gr, S);
  grad_global<ALIGNED, T, CAP>(xr + col_beg, dr + col_beg, col_end - col_beg, map, S);
  if constexpr (!TOPK) {
    if (id >= col_beg && id < col_end) {
      __syncthreads();
      if (threadIdx.x == 0) Out8<T>::store1(dr + id, map.at(load1(xr + id), gr.G, gr, S));
    }
  } else {
    __syncthreads();
    grad_targets<T, CAP>(dr, t, s_n, map, gr, S);
  }
}

template <class T, int LOSS, bool CAP, bool STAGED, bool ALIGNED, bool MANY = false>
cudaError_t launch_loss_t(const LossArgs& a, cudaStream_t s) {
  if constexpr (LOSS == kLossDistill && !MANY) {
    if (a.k > kFewTargets) return launch_loss_t<T, LOSS, CAP, STAGED, ALIGNED, true>(a, s);
  }
  const auto kernel = row_loss_kernel<T, LOSS, CAP, STAGED, ALIGNED, MANY>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows * a.cluster));
  cfg.blockDim = dim3(row_threads<LOSS>());
  cfg.dynamicSmemBytes = (LOSS == kLossDistill ? target_smem(a.k) : 0) + (STAGED ? stage_bytes<T>(8 * a.vec_per_cta) : 0);
  cfg.stream = s;
  if (LOSS != kLossLogp) {
    // once per device: more dynamic shared memory and larger clusters than the defaults
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLossMaxSmem);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
    }
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Every row of the logits (and of the gradient, whose rows follow one another)
// starts on a 16-byte boundary: the kernels without the other path need fewer
// registers and instructions.
template <class T>
bool rows_aligned(const void* x, const vls_rows& r, const void* dx, int64_t V) {
  constexpr int64_t per = 16 / sizeof(T);
  return ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dx)) & 15u) == 0 && r.ld % per == 0 &&
         r.ld_group % per == 0 && (dx == nullptr || V % per == 0);
}

template <class T, int LOSS, bool CAP>
cudaError_t launch_loss_staged(const LossArgs& a, cudaStream_t s) {
  const bool al = rows_aligned<T>(a.x, a.rx, a.dx, a.vocab);
  if constexpr (LOSS == kLossLogp) {
    return al ? launch_loss_t<T, LOSS, CAP, false, true>(a, s) : launch_loss_t<T, LOSS, CAP, false, false>(a, s);
  } else {
    if (!a.staged) return launch_loss_t<T, LOSS, CAP, false, false>(a, s);
    return al ? launch_loss_t<T, LOSS, CAP, true, true>(a, s) : launch_loss_t<T, LOSS, CAP, true, false>(a, s);
  }
}

template <int LOSS>
cudaError_t launch_loss_op(vls_dtype dt, bool cap, const LossArgs& a, cudaStream_t s) {
  if (dt == VLS_BF16)
    return cap ? launch_loss_staged<__nv_bfloat16, LOSS, true>(a, s) : launch_loss_staged<__nv_bfloat16, LOSS, false>(a, s);
  if (dt == VLS_F16)
    return cap ? launch_loss_staged<__half, LOSS, true>(a, s) : launch_loss_staged<__half, LOSS, false>(a, s);
  return cap ? launch_loss_staged<float, LOSS, true>(a, s) : launch_loss_staged<float, LOSS, false>(a, s);
}

}  // namespace vls
