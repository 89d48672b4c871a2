"""Corners of the training losses, where a call's answer is easily wrong or
refused.  The helpers and tolerances are those of test_losses.py."""

import math

import numpy as np
import pytest
import torch

import loss_reference as ref
import vocab_log_softmax_gb300 as vls
from test_losses import CFG, DEV, DTYPES, INF, _check_distill, _check_policy, _check_preference, _distill_inputs, _gen
from test_losses import _logits, _np, _policy_inputs, _preference_inputs
from vls_compare import assert_grad_close, bitwise_equal, to_f64
from vocab_log_softmax_gb300 import _lib, build
from vocab_log_softmax_gb300 import binding as B

gpu = pytest.mark.gpu
NAN = float("nan")
P = 0x1000   # non-NULL, never dereferenced


# ---------------------------------------------------------------------------
# label smoothing
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kind", ["hinge", "squared"])
def test_label_smoothing_of_the_other_kinds(kind):
    """The hinge and the squared loss have no smoothing: a call that passes one
    (one training configuration for every kind) gets the loss as it is.  A value
    outside [0, 1/2) stays refused."""
    gen = _gen(1)
    x = _logits(7, 515, "bf16", gen)
    ids, offsets, rf, w, margin = _preference_inputs(x, [3, 4], gen)
    want = B.vls_preference_loss(x, ids, offsets, rf, w, margin, kind=kind)
    got = B.vls_preference_loss(x, ids, offsets, rf, w, margin, kind=kind, label_smoothing=0.1)
    for key in want:
        assert bitwise_equal(want[key], got[key]), key
    a = vls.preference_loss(x, ids, offsets, ref_logp=rf, weights=w, margin=margin, kind=kind, label_smoothing=0.1)
    assert bitwise_equal(a[1], want["pair_loss"])
    for wrong in (0.5, -0.1, NAN):
        with pytest.raises(ValueError):
            B.vls_preference_loss(x, ids, offsets, kind=kind, label_smoothing=wrong)


def test_label_smoothing_reaches_the_sigmoid_loss_alone():
    for kind, code in (("sigmoid", 0), ("hinge", 1), ("squared", 2)):
        cfg = B._pref_cfg(kind, True, 0.25, 0.125)
        assert (cfg.kind, cfg.length_average, cfg.beta) == (code, 1, 0.25)
        assert cfg.label_smoothing == (0.125 if kind == "sigmoid" else 0.0)
        assert B._pref_cfg(kind, False, 0.25, 0.5).label_smoothing == 0.5      # for the library to refuse


# ---------------------------------------------------------------------------
# distillation: large teacher logits under a temperature
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("k", [16, 64, 65, 300])
@pytest.mark.parametrize("tau", [float(np.float32(0.7)), 1.5])
@pytest.mark.parametrize("offset", [0.0, 100.0, 1000.0, -8192.0])
def test_teacher_offset_under_a_temperature(offset, tau, k, lse):
    """A common offset of the teacher's logits moves no probability by more than
    the rounding of their differences: those are multiples of 1/64 below 32, so
    exact in fp32, and their scaling by 1/tau is off by 2^-23 of at most 32 / 0.7
    (6e-6 at an exponent of 46, whose probability is below 1e-20; 2e-6 at the
    exponents of up to 15 that matter).  With the teacher's log-sum-exp the
    largest logit's gap to it is one rounded difference, of a few units."""
    gen = _gen(k)
    x = _logits(4, 5000, "fp32", gen)
    ids, t, w, _ = _distill_inputs(x, k, gen, distinct=True)
    t = (t * 64).round() / 64 + offset
    ls = None
    if lse:
        more = torch.tensor([0.1, 0.7, 1.3, 2.1], dtype=torch.float64, device=DEV)
        ls = (torch.logsumexp(t.double() / tau, 1) + more).float()
    out = B.vls_distill_loss(x, ids, t, w, ls, temperature=tau)
    _check_distill(x, ids, t, w, ls, out, tau=tau, what=f"offset {offset}")


@gpu
@pytest.mark.parametrize("lse", [False, True])
def test_teacher_rows_without_mass(lse):
    """Teacher entries that are all -inf: without the log-sum-exp they have no
    distribution (NaN); with it every probability is 0, and so are the loss and
    the gradient."""
    gen = _gen(14)
    for k, v in ((5, 2003), (70, 2003), (5, 70001), (70, 70001)):
        x = _logits(3, v, "fp32", gen)
        ids, t, w, ls = _distill_inputs(x, k, gen, 0.5, lse, distinct=True)
        t[1] = -INF
        t[2, 1:] = -INF
        out = B.vls_distill_loss(x, ids, t, w, ls, temperature=0.5)
        _check_distill(x[::2], ids[::2], t[::2], w[::2], ls[::2] if lse else None,
                       B.vls_distill_loss(*(a[::2].contiguous() if a is not None else None
                                            for a in (x, ids, t, w, ls)), temperature=0.5), tau=0.5)
        if lse:
            assert out["row_loss"][1] == 0 and torch.count_nonzero(out["coef"][1]) == 0
            assert torch.count_nonzero(out["dlogits"][1]) == 0
        else:
            assert torch.isnan(out["row_loss"][1]) and torch.isnan(out["coef"][1]).all()
            assert torch.isnan(out["dlogits"][1]).all()


# ---------------------------------------------------------------------------
# NaN among a loss's constants
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("kl", [False, True])
@pytest.mark.parametrize("dual", [0.0, 3.0])
def test_policy_nan_constants(dtype, kl, dual):
    """A NaN old_logp or advantage makes the token's loss NaN; its coefficient
    and gradient row are NaN with it, wherever the ratio lies, and the other
    rows keep their bits.  At an ignored id the constants are not looked at."""
    gen = _gen(19)
    n, v = 10, 1031
    x = _logits(n, v, dtype, gen)
    ids, old, adv, w, rf = _policy_inputs(x, gen, ignore=False)
    rf = rf if kl else None
    kw = dict(clip_low=0.2, clip_high=0.3, dual_clip=dual, kl_coef=0.05 if kl else 0.0)
    ids[9] = -100
    base = B.vls_policy_loss(x, ids, old, adv, w, rf, **kw)
    logp = base["logp"]
    old, adv = old.clone(), adv.clone()
    old[0] = NAN
    for i, step in ((1, 0.0), (2, 2.0), (3, -2.0), (4, 0.1)):     # ratios inside, above and below the clip range
        old[i] = logp[i] - step
        adv[i] = NAN
    old[9] = adv[9] = NAN
    out = B.vls_policy_loss(x, ids, old, adv, w, rf, **kw)
    for i in range(5):
        assert torch.isnan(out["row_loss"][i]) and torch.isnan(out["coef"][i]), i
        assert torch.isnan(out["dlogits"][i]).all(), i
    assert torch.isnan(out["loss"])
    for key in ("row_loss", "logp", "coef", "dlogits"):
        assert bitwise_equal(out[key][5:], base[key][5:]), key
    again = B.vls_loss_bwd(x, ids, out["coef"], out["stats"])
    assert torch.isnan(again[:5]).all() and bitwise_equal(again[5:], out["dlogits"][5:])


@gpu
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("where", ["margin", "ref", "logits"])
def test_preference_nan(kind, where):
    """A NaN in a pair makes its loss NaN and the gradient of every valid row of
    the pair; the other pair keeps its bits."""
    gen = _gen(23)
    lengths = [4, 3, 5, 2]          # pairs (0, 2), (1, 3)
    x = _logits(sum(lengths), 1031, "fp32", gen)
    ids, offsets, rf, w, margin = _preference_inputs(x, lengths, gen)
    ids[1] = -100
    kw = dict(kind=kind, beta=0.5)
    base = B.vls_preference_loss(x, ids, offsets, rf, w, margin, **kw)
    x, rf, margin = x.clone(), rf.clone(), margin.clone()
    if where == "margin":
        margin[0] = NAN
    elif where == "ref":
        rf[2] = NAN
    else:
        x[2, 7] = NAN
    out = B.vls_preference_loss(x, ids, offsets, rf, w, margin, **kw)
    first = [0, 2, 3] + list(range(7, 12))
    second = list(range(4, 7)) + [12, 13]
    assert torch.isnan(out["pair_loss"][0]) and torch.isnan(out["coef"][first]).all()
    assert torch.isnan(out["dlogits"][first]).all()
    assert torch.count_nonzero(out["dlogits"][1]) == 0 and out["coef"][1] == 0
    for key in ("logp", "coef", "dlogits"):
        assert bitwise_equal(out[key][second], base[key][second]), key
    assert bitwise_equal(out["pair_loss"][1:], base["pair_loss"][1:])


@gpu
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
def test_preference_infinities(kind):
    """A target of probability 0, masked columns and columns of the type's lowest
    value: the rewards are infinite where the definition's are, u is infinite on
    the right and on the wrong side, and no finite row has a NaN."""
    gen = _gen(24)
    lengths = [3, 3, 3, 3, 3, 3]     # pairs (0, 3), (1, 4), (2, 5)
    x = _logits(18, 1031, "bf16", gen)
    ids, offsets, rf, w, _ = _preference_inputs(x, lengths, gen)
    x[0, : 1031 // 2] = torch.finfo(torch.bfloat16).min
    ids[0] = 1030
    x[4, ::3] = -INF
    ids[4] = 1
    rf[0] = rf[4] = -5.0
    x[7, ids[7]] = -INF              # pair 2: the preferred one has probability 0
    x[12, ids[12]] = -INF            # pair 1: the other one has
    out = B.vls_preference_loss(x, ids, offsets, rf, w, kind=kind, beta=0.5)
    with np.errstate(all="ignore"):
        r = ref.preference(to_f64(x), _np(ids), _np(offsets), _np(rf), None, _np(w), kind, 0.5)
    for key in ("logp", "pair_loss", "reward"):
        got, want = _np(out[key]), r[key]
        assert np.array_equal(np.isinf(got), np.isinf(want)) and not np.isnan(got).any(), key
        assert np.array_equal(got[np.isinf(got)], want[np.isinf(want)]), key
    fine = np.isfinite(r["coef"])
    assert np.array_equal(np.isfinite(_np(out["coef"])), fine)
    g = ref.grad_rows(to_f64(x), _np(ids)[:, None], _np(out["coef"])[:, None])
    assert_grad_close(out["dlogits"][torch.tensor(fine)], g[fine], "dlogits")


@gpu
def test_policy_zero_advantage_beyond_fp32():
    """A ratio that overflows fp32 (log-probability 100 above the recorded one)
    times an advantage of 0 is 0, as in the definition; with a recorded
    probability of 0 the ratio is infinite and 0 times it is NaN."""
    x = torch.zeros((4, 2), device=DEV)
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    old = torch.tensor([-100.0, -100.0, -INF, -100.0], device=DEV)
    adv = torch.tensor([0.0, -0.0, 0.0, 1.0], device=DEV)
    for dual in (0.0, 3.0):
        out = B.vls_policy_loss(x, ids, old, adv, None, None, dual_clip=dual)
        assert out["row_loss"][:2].tolist() == [0.0, 0.0] and out["coef"][:2].tolist() == [0.0, 0.0]
        assert torch.count_nonzero(out["dlogits"][:2]) == 0
        assert torch.isnan(out["row_loss"][2]) and torch.isnan(out["coef"][2])
        assert abs(out["row_loss"][3].item() + 1.2) < 1e-6 and out["coef"][3] == 0


# ---------------------------------------------------------------------------
# preference: rows outside every sequence
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("v", [1031, 70000])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_rows_outside_every_sequence(dtype, v, cap):
    """The rows before the first sequence and behind the last take no part
    whatever they hold (a buffer's unused end): valid ids on logits that are NaN,
    infinite or all -inf get a gradient of exactly 0, from the call and from its
    statistics."""
    gen = _gen(25)
    lengths = [4, 3]
    x = _logits(2 + sum(lengths) + 5, v, dtype, gen)
    ids, offsets, rf, w, margin = _preference_inputs(x, lengths, gen, lead=2, cap=cap)
    base = B.vls_preference_loss(x, ids, offsets, rf, w, margin, cap=cap)
    x = x.clone()
    x[0] = NAN
    x[1, 3] = INF
    x[9] = -INF
    x[10, 0] = NAN
    x[11] = INF
    x[12, 1:] = -INF
    out = B.vls_preference_loss(x, ids, offsets, rf, w, margin, cap=cap)
    inside, outside = slice(2, 9), [0, 1] + list(range(9, 14))
    for key in ("loss", "pair_loss", "reward"):
        assert bitwise_equal(out[key].reshape(-1), base[key].reshape(-1)), key
    for key in ("logp", "coef", "dlogits"):
        assert bitwise_equal(out[key][inside], base[key][inside]), key
    assert torch.equal(out["coef"][outside], torch.zeros(7, device=DEV))
    assert torch.equal(out["dlogits"][outside], torch.zeros_like(out["dlogits"][outside]))
    for up in (1.0, -0.37):
        again = B.vls_loss_bwd(x, ids, out["coef"], out["stats"], torch.tensor(up, device=DEV), cap=cap)
        assert torch.equal(again[outside], torch.zeros_like(again[outside]))
        assert torch.isfinite(again[inside]).all()
    leaf = x.clone().requires_grad_(True)
    (3.0 * vls.preference_loss(leaf, ids, offsets, ref_logp=rf, softcap=cap or None)[0]).backward()
    assert torch.equal(leaf.grad[outside], torch.zeros_like(leaf.grad[outside]))


@gpu
def test_one_column_rows_keep_their_gradient():
    """Rows whose statistics are those of a row without a target (max 0, log-sum
    0): one column, or one column that holds all the mass."""
    x = torch.tensor([[0.0, -200.0], [0.0, -200.0], [0.0, -200.0]], device=DEV)
    ids = torch.tensor([0, 1, 1], device=DEV)
    offsets = torch.tensor([0, 1, 3], device=DEV)
    for kind in ("sigmoid", "squared"):     # u = 100: the coefficients are 2e-44 and 398
        out = B.vls_preference_loss(x, ids, offsets, torch.full((3,), -200.0, device=DEV), kind=kind, beta=0.5)
        assert _np(out["stats"]).tolist() == [[0.0, 0.0]] * 3
        g = ref.grad_rows(to_f64(x), _np(ids)[:, None], _np(out["coef"])[:, None])
        assert_grad_close(out["dlogits"], g)
    assert torch.count_nonzero(out["coef"]) == 3 and torch.count_nonzero(out["dlogits"][1:]) == 4


# ---------------------------------------------------------------------------
# distillation with more than 64 targets: kernels of their own
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("cap,tau", [(0.0, 1.0), (0.0, 2.0), (30.0, 1.0), (30.0, 0.5)])
@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("k,v", [(70, 30011), (300, 30011), (70, 151936), (1024, 151937)])
def test_distill_forms_of_many_targets(dtype, cap, tau, lse, k, v):
    gen = _gen(k + v)
    x = _logits(3, v, dtype, gen, 5.0)
    args = _distill_inputs(x, k, gen, tau, lse, distinct=True)
    out = B.vls_distill_loss(x, *args, cap=cap, temperature=tau)
    _check_distill(x, *args, out, cap, tau)


@gpu
@pytest.mark.parametrize("tdt", sorted(DTYPES))
@pytest.mark.parametrize("lse", [False, True])
@pytest.mark.parametrize("k,v", [(12, 70001), (65, 2003), (70, 70001), (513, 70000)])
def test_many_targets_ragged_rows_and_masks(tdt, lse, k, v):
    """As test_distill_ragged_rows_and_masks, on rows of one CTA and of several."""
    gen = _gen(29)
    n = 10
    x = _logits(n, v, "bf16", gen)
    ids, t, w, ls = _distill_inputs(x, k, gen, 1.0, lse)
    t = t.to(DTYPES[tdt])
    ids[0, 4:] = -100
    ids[1, :] = -100
    ids[2, :] = 77
    ids[3, ::2] = v
    t[4, :5] = -INF
    x[5, ids[5, 0]] = -INF
    ids[5, 1:] = torch.arange(1, k, device=DEV) + 5 + ids[5, 0] % 900
    t[6, 0] = -INF
    ids[6] = torch.arange(k, device=DEV) * 3
    x[6, 0] = -INF
    x[7, :] = -INF
    x[8, 3] = NAN
    x[9, :] = -INF
    ids[9, :] = -1
    out = B.vls_distill_loss(x, ids, t, w, ls)
    r = _check_distill(x, ids, t, w, ls, out)
    assert np.isposinf(r["row_loss"][5]) and np.isnan(r["row_loss"][7]) and np.isnan(r["row_loss"][8])
    assert np.isfinite(r["row_loss"][6]) and r["row_loss"][1] == 0 and r["row_loss"][9] == 0
    for i in (1, 9):
        assert torch.count_nonzero(out["dlogits"][i]) == 0 and torch.count_nonzero(out["coef"][i]) == 0
    g = B.vls_loss_bwd(x, ids, out["coef"], out["stats"])
    fine = [0, 1, 2, 3, 4, 5, 6, 9]
    assert_grad_close(g[fine], to_f64(out["dlogits"])[fine], "again")


@gpu
@pytest.mark.parametrize("k", [9, 70, 300])
def test_many_targets_invariance(k):
    """Bits do not depend on the layout, on the other rows, on a repetition or on
    whether the gradient is asked for."""
    gen = _gen(30)
    x = _logits(20, 70003, "bf16", gen)
    args = _distill_inputs(x, k, gen, 0.7, True)
    kw = dict(temperature=0.7)
    full = B.vls_distill_loss(x, *args, **kw)
    wide = torch.full((20, 70003 + 13), 5.0, dtype=x.dtype, device=DEV)
    wide[:, :70003] = x
    quiet = B.vls_distill_loss(x, *args, grad=False, **kw)
    for key in full:
        assert bitwise_equal(full[key], B.vls_distill_loss(wide[:, :70003], *args, **kw)[key]), key
        assert key == "dlogits" or bitwise_equal(full[key], quiet[key]), key
    p = torch.tensor([19, 3, 11], device=DEV)
    part = B.vls_distill_loss(x[p], *(a[p].contiguous() for a in args), **kw)
    for key in ("row_loss", "coef", "stats", "dlogits"):
        assert bitwise_equal(full[key][p], part[key]), key


@gpu
@pytest.mark.parametrize("dtype,v", [("bf16", 1638400), ("bf16", 1638399), ("bf16", 1638401), ("fp32", 819200),
                                     ("fp32", 819201)])
def test_longest_staged_rows(dtype, v):
    """Rows that fill the shared memory of the largest cluster, with the most
    targets beside them, and rows one column longer."""
    gen = _gen(v)
    x = _logits(2, v, dtype, gen)
    args = _policy_inputs(x, gen)
    _check_policy(x, *args, B.vls_policy_loss(x, *args, **CFG), what="policy")
    for k in (64, 1024):
        d = _distill_inputs(x, k, gen)
        _check_distill(x, *d, B.vls_distill_loss(x, *d), what=f"distill k={k}")


# ---------------------------------------------------------------------------
# shapes of the constants, temperatures
# ---------------------------------------------------------------------------

def test_constants_of_another_shape():
    """[T, B] constants beside [B, T, V] logits would be taken in the wrong
    order.  The leading dimensions' shape, one flattened dimension and shapes that
    differ by dimensions of size 1 say the same order."""
    b, t, v = 2, 3, 6
    x, i = torch.zeros((b, t, v)), torch.zeros((b, t), dtype=torch.int64)
    f, wrong = torch.zeros((b, t)), torch.zeros((t, b))
    for kw in (dict(old_logp=wrong, advantages=f), dict(old_logp=f, advantages=wrong),
               dict(old_logp=f, advantages=f, ref_logp=wrong), dict(old_logp=f, advantages=f, weights=wrong)):
        with pytest.raises(ValueError, match="shape"):
            vls.policy_loss(x, i, **kw)
    for kw in (dict(teacher_lse=wrong), dict(weights=wrong)):
        with pytest.raises(ValueError, match="shape"):
            vls.distill_loss(x, i[..., None], f[..., None], **kw)
    y, j, g = torch.zeros((6, 2, v)), torch.zeros((6, 2), dtype=torch.int64), torch.zeros((2, 6))
    with pytest.raises(ValueError, match="shape"):
        vls.preference_loss(y, j, ref_logp=g)
    values = torch.arange(6.0)
    for shape in ((2, 3), (6,), (2, 3, 1), (1, 2, 3), (2, 1, 3)):
        assert vls._const(values.view(shape), torch.Size((2, 3)), "a").tolist() == values.tolist()
    assert vls._const(values.view(2, 3), values.shape, "a").tolist() == values.tolist()    # flattened logits
    assert vls._const(torch.ones(()), torch.Size(()), "a").tolist() == [1.0]
    assert vls._const(None, torch.Size((2, 3)), "a") is None
    for shape in ((3, 2), (5,), (1, 6, 2)):
        with pytest.raises(ValueError):
            vls._const(torch.zeros(shape), torch.Size((2, 3)), "a")


def test_temperatures_whose_exponents_overflow():
    """log2(e) / temperature, and 2 cap log2(e) / temperature with a softcap, have
    to be fp32 numbers; smaller temperatures are refused by every call."""
    build.build()
    tlib = _lib.load_test()
    assert tlib.vls_test_set_fault(_lib.VLS_TEST_FAULT_DEVICE) == 0
    rows = _lib.rows(10)

    def calls(cap, tau):
        cfg = _lib.VlsPolicyCfg(0.2, 0.2, 0.0, 0.0)
        yield tlib.vls_policy_loss(P, rows, 1, 4, 10, P, -100, cap, tau, cfg, P, P, None, None, P, P, P, P, P, P, None)
        yield tlib.vls_distill_loss(P, rows, 1, 4, 10, P, 3, -100, cap, tau, P, 0, None, None, P, P, P, P, P, None)
        yield tlib.vls_loss_bwd(P, rows, 1, 4, 10, P, 1, -100, cap, tau, P, P, None, 0, P, None)

    try:
        for cap, tau, code in ((0.0, 3.5e-39, 7), (0.0, 4.5e-39, 5), (30.0, 2.0e-37, 7), (30.0, 3.0e-37, 5),
                               (1e30, 1e-9, 7), (1e30, 1e-7, 5), (0.0, 1e-3, 5), (0.0, 3e38, 5), (30.0, 1.0, 5)):
            assert list(calls(cap, tau)) == [code] * 3, (cap, tau)
    finally:
        tlib.vls_test_set_fault(_lib.VLS_TEST_FAULT_NONE)
