"""Rows that hold whole runs of one value: columns masked in one of two
tensors only (a policy restricted to some columns beside an unrestricted
reference), so that a thread's first vectors are -inf on one side and finite on
the other.  Against the oracle, at the plain rules."""

import numpy as np
import pytest
import torch

import oracle
from test_parity_configs import check_entropy, check_kl, check_logp
from vls_compare import assert_fp32_close, assert_grad_close, bitwise_equal, to_f64, ulp_bf16, ulp_f16
from vocab_log_softmax_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [9, 257, 4099, 16384, 65537, 262147]
# columns set to one value: the runs of a row (start, end; negative: from the end)
RUNS = [(0, 8), (8, 16), (0, 64), (0, 2048), (2048, 4096), (-3, None), (-16, None), (0, -1), (1, -1)]


def _data(v, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = len(RUNS) + 2
    a = (3.0 * torch.randn((n, v), generator=g, device=DEV)).to(dtype)
    b = (a.float() + 0.5 * torch.randn((n, v), generator=g, device=DEV)).to(dtype)
    ids = torch.randint(0, v, (n, 3), generator=g, device=DEV)
    return a, b, ids, torch.randn((n, 3), generator=g, device=DEV), torch.randn((n,), generator=g, device=DEV)


def _fill(x, value):
    """Row i: run i of RUNS; the row behind them: every other vector of 8 columns; the last row: as it is."""
    for i, (s, e) in enumerate(RUNS):
        x[i, s:e] = value
    for c in range(0, x.shape[1], 16):
        x[len(RUNS), c:c + 8] = value
    return x


def _capped_grad_close(got, want, x, weight, cap, what):
    """The gradient rule with the capped logits' own rounding in its bound.  z =
    c - 2 c r with r = 1 / (1 + 2^t): the exponential is off by 2^-22 and the
    reciprocal by 2^-23 of itself, so z by at most 2 c (2^-22 + 2^-23), and a
    difference of two of them by twice that.  The gradients p (log p - ...) and
    onehot - p carry it times p and the upstream weight: a row with almost all its
    mass in one column, where p is 1 and the true gradient 0, has nothing else."""
    z = cap * np.tanh(x / cap)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    g = to_f64(got)
    if got.dtype == torch.float32:
        rule = 1e-5 + 1e-5 * np.abs(want)
    else:
        rule = (ulp_bf16 if got.dtype == torch.bfloat16 else ulp_f16)(want) + 1e-6
    over = np.abs(g - want) - rule - weight[:, None] * p * (2 * 2 * cap * (2.0 ** -22 + 2.0 ** -23))
    assert np.isfinite(want).all() and np.isfinite(g).all(), what
    assert (over <= 0).all(), (what, np.unravel_index(over.argmax(), over.shape), over.max())


def _check_capped(a, b, ids, gk, gr, direction, cap, what):
    """check_kl, check_entropy and check_logp with that bound; returns the KL."""
    xa, xb, g, i = to_f64(a), to_f64(b), to_f64(gr), ids.cpu().numpy()
    kl, sa, sb = B.vls_kl_fwd(a, b, direction, cap)
    assert_fp32_close(kl, oracle.kl_fwd(xa, xb, direction, cap), f"{what} {direction} fwd")
    _capped_grad_close(B.vls_kl_bwd(a, b, gr, kl, sa, sb, direction, cap), oracle.kl_bwd(xa, xb, g, direction, cap), xa,
                       np.abs(g), cap, f"{what} {direction}")
    H, st = B.vls_entropy_fwd(a, cap)
    assert_fp32_close(H, oracle.entropy_fwd(xa, cap), f"{what} entropy")
    _capped_grad_close(B.vls_entropy_bwd(a, gr, H, st, cap), oracle.entropy_bwd(xa, g, cap), xa, np.abs(g), cap,
                       f"{what} entropy")
    lp, st = B.vls_logp_fwd(a, ids, -100, cap)
    assert_fp32_close(lp, oracle.logp_fwd(xa, i, -100, cap), f"{what} logp")
    _capped_grad_close(B.vls_logp_bwd(a, ids, gk, st, -100, cap), oracle.logp_bwd(xa, i, to_f64(gk), -100, cap), xa,
                       np.abs(to_f64(gk)).sum(1), cap, f"{what} logp")
    return kl


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", SIZES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_kl_of_a_masked_side(v, dtype, cap):
    """KL(P || Q) with P masked over whole runs where Q is finite is finite; with
    Q masked it is +inf (with a cap, where no logit stays -inf, finite).  The
    fused call agrees, and its entropy and log-probabilities are a's own."""
    a, b, ids, gk, gr = _data(v, dtype, v)
    _fill(a, -INF)
    for d in ("reverse", "forward"):
        for x, y in ((a, b), (b, a)):
            if cap:
                kl = _check_capped(x, y, ids, gk, gr, d, cap, f"V={v}")
            else:
                kl = check_kl(x, y, gr, d, what=f"V={v}")
            out = B.vls_fused_fwd(x, y, ids, direction=d, cap=cap)
            H, _ = B.vls_entropy_fwd(x, cap)
            lp, _ = B.vls_logp_fwd(x, ids, -100, cap)
            assert bitwise_equal(out["kl"], kl) and bitwise_equal(out["H"], H) and bitwise_equal(out["logp"], lp)
    if not cap:
        check_entropy(a, gr, what="entropy")
        check_logp(a, ids, gk, what="logp")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("direction", ["reverse", "forward"])
def test_kl_of_a_masked_side_sharded(dtype, direction):
    """The same over shards of the vocabulary, one of them masked throughout."""
    v = 40000
    a, b, *_ = _data(v, dtype, 3)
    _fill(a, -INF)
    a[1, 10000:20000] = -INF
    for x, y in ((a, b), (b, a)):
        parts = torch.stack([B.vls_kl_partial(x[:, s:e], y[:, s:e], direction)
                             for s, e in ((0, 10000), (10000, 20000), (20000, v))])
        kl, _, _ = B.vls_kl_combine(parts, direction)
        assert_fp32_close(kl, oracle.kl_fwd(to_f64(x), to_f64(y), direction), "sharded kl")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("direction", ["reverse", "forward"])
def test_fused_gradient_of_a_masked_side(dtype, direction):
    a, b, ids, gl, gr = _data(4099, dtype, 5)
    _fill(a if direction == "reverse" else b, -INF)
    out = B.vls_fused_fwd(a, b, ids, direction=direction)
    d = B.vls_fused_bwd(a, out, b, ids, g_logp=gl, g_H=gr, g_kl=gr, direction=direction)
    xa, xb = to_f64(a), to_f64(b)
    ref = (oracle.logp_bwd(xa, ids.cpu().numpy(), gl.cpu().numpy()) + oracle.entropy_bwd(xa, gr.cpu().numpy())
           + oracle.kl_bwd(xa, xb, gr.cpu().numpy(), direction))
    assert_grad_close(d, ref, "fused gradient")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", SIZES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_runs_of_nan(v, dtype, cap):
    """A NaN logit makes every statistic and gradient of its row NaN, whole
    vectors and whole warps' shares of nothing else among them; the last row (and
    one whose run lies behind a short row's end) is finite."""
    a, b, ids, gk, gr = _data(v, dtype, v + 1)
    _fill(a, float("nan"))
    n, nan = len(a), torch.isnan(a).any(1)
    assert nan.sum() >= n - 2 and not nan[-1]
    H, st = B.vls_entropy_fwd(a, cap)
    lp, sl = B.vls_logp_fwd(a, ids, -100, cap)
    grads = [B.vls_entropy_bwd(a, gr, H, st, cap), B.vls_logp_bwd(a, ids, gk, sl, -100, cap)]
    stats = [H, lp, st, sl]
    for d in ("reverse", "forward"):
        for x, y in ((a, b), (b, a)):
            kl, sx, sy = B.vls_kl_fwd(x, y, d, cap)
            grads.append(B.vls_kl_bwd(x, y, gr, kl, sx, sy, d, cap))
            out = B.vls_fused_fwd(x, y, ids, direction=d, cap=cap)
            stats += [kl, out["kl"]] + ([out["H"], out["logp"]] if x is a else [])
    for i, s in enumerate(stats):
        s = s.reshape(n, -1)
        s = s[:, 1:] if i in (2, 3) else s      # (max, log-sum): the max is that of the columns that are numbers
        assert torch.isnan(s[nan]).all() and torch.isfinite(s[~nan]).all(), i
    for i, d in enumerate(grads):
        assert torch.isnan(d[nan]).all() and torch.isfinite(d[~nan]).all(), i


@pytest.mark.parametrize("dtype", DTYPES)
def test_runs_of_nan_sharded(dtype):
    """A shard of nothing but NaN among finite ones."""
    v = 30000
    a, b, ids, *_ = _data(v, dtype, 4)
    a[0, 10000:20000] = float("nan")
    a[1, :10000] = float("nan")
    a[2, 12000:12008] = float("nan")
    bounds = ((0, 10000), (10000, 20000), (20000, v))
    both = [B.vls_logp_partial(a[:, s:e], ids, s, v) for s, e in bounds]
    lp, _ = B.vls_logp_combine(torch.stack([p for p, _ in both]), torch.stack([z for _, z in both]), ids, v)
    H, _ = B.vls_entropy_combine(torch.stack([B.vls_entropy_partial(a[:, s:e]) for s, e in bounds]))
    outs = [lp, H]
    for d in ("reverse", "forward"):
        for x, y in ((a, b), (b, a)):
            outs.append(B.vls_kl_combine(torch.stack([B.vls_kl_partial(x[:, s:e], y[:, s:e], d) for s, e in bounds]), d)[0])
    for o in outs:
        assert torch.isnan(o[:3]).all() and torch.isfinite(o[3:]).all()


@pytest.mark.parametrize("start,end", [(0, 32), (0, 64), (32, 96), (0, 2048), (2048, 2100), (3, 2990)])
def test_linear_head_runs_of_nan(start, end):
    """Rows of the head's weight that are NaN make their columns NaN, and with them
    every row's statistics, whatever run of columns they fill."""
    g = torch.Generator(device=DEV).manual_seed(7)
    h = torch.randn((130, 72), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((3000, 72), generator=g, device=DEV).to(torch.bfloat16)
    ids = torch.full((130, 1), 2999, device=DEV)
    base, _, _ = B.vls_linear_logp_fwd(h, w, ids)
    assert torch.isfinite(base).all()
    w[start:end] = float("nan")
    lp, st, status = B.vls_linear_logp_fwd(h, w, ids)
    lp2, _, status2 = B.vls_linear_logp_fwd_noalloc(h, w, ids)
    assert int(status.item()) == 0 and int(status2.item()) == 0
    assert torch.isnan(lp).all() and torch.isnan(lp2).all() and torch.isnan(st[:, 1]).all()
    one = h.clone()
    one[5] = float("nan")
    lp, _, _ = B.vls_linear_logp_fwd(one, torch.nan_to_num(w), ids)
    assert torch.isnan(lp[5]).all() and torch.isfinite(lp[:5]).all() and torch.isfinite(lp[6:]).all()
