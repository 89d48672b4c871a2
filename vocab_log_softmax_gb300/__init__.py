"""vocab_log_softmax_gb300: row-wise vocabulary log-softmax statistics on
GB300 (sm_103a).

Two layers over the CUDA library libvls (C ABI in include/vls.h):

* ``binding``: ``vls_*`` functions with the C ABI's names, argument
  marshalling only (tensors in, raw pointers to the library);
* the autograd functions below -- ``logprobs``, ``entropy``, ``kl`` and
  ``softcap`` -- which save the forward's per-row statistics so that each
  backward is one read of the logits and one write of the gradient; and the
  training losses ``policy_loss``, ``distill_loss`` and ``preference_loss``,
  whose forward makes the gradient of the logits as well.

Every computation runs in the library's kernels; there is no CPU or eager
fallback, and a missing library raises.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._lib import VlsArgumentError, VlsDeviceError, VlsError  # noqa: F401
from .binding import (  # noqa: F401
    vls_check_device_error,
    vls_distill_loss,
    vls_loss_bwd,
    vls_policy_loss,
    vls_preference_loss,
    vls_linear_logp_bwd,
    vls_linear_logp_fwd,
    vls_entropy_bwd,
    vls_entropy_fwd,
    vls_fused_bwd,
    vls_fused_fwd,
    vls_kl_bwd,
    vls_kl_fwd,
    vls_logp_bwd,
    vls_logp_fwd,
    vls_softcap_bwd,
    vls_softcap_fwd,
    vls_status_string,
    vls_version,
)

__all__ = ["logprobs", "entropy", "kl", "softcap", "stats", "linear_logprobs", "policy_loss", "distill_loss",
           "preference_loss", "check_device_error"]


def check_device_error() -> None:
    """Raises VlsDeviceError if a bounded wait of a tensor-core kernel ran out
    on the current device since the last check (synchronises the device)."""
    vls_check_device_error()


def _addressable(rows: torch.Tensor) -> bool:
    """Whether the kernels can read a [N, V] or [B, T, V] view in place: every
    row stride at least V (broadcast rows, for one, are not)."""
    v = rows.shape[-1]
    return all(size <= 1 or stride >= v for size, stride in zip(rows.shape[:-1], rows.stride()[:-1]))


def _as_rows(x: torch.Tensor) -> torch.Tensor:
    """[..., V] -> a [N, V] view, or a [B, T, V] view read with two row strides
    (a slice such as ``x[:, :-1]`` stays in place); layouts the kernels cannot
    address, such as a strided vocabulary dimension, are copied first."""
    if x.dim() == 0:
        raise ValueError("expected at least one dimension (the vocabulary)")
    v = x.shape[-1]
    if x.dim() == 1:
        x = x.reshape(1, v)
    if v > 1 and x.stride(-1) != 1:
        x = x.contiguous()
    try:
        rows = x.view(-1, v)
    except RuntimeError:
        try:
            rows = x.view(-1, x.shape[-2], v)
        except RuntimeError:
            rows = x.reshape(-1, v)
    return rows if _addressable(rows) else rows.contiguous()


def _nrows(rows: torch.Tensor) -> int:
    return rows.shape[:-1].numel()


def _ids_rows(ids: torch.Tensor, n: int) -> torch.Tensor:
    """ids shaped like the logits' leading dims (k = 1) or with a trailing k -> [N, k] int64."""
    if n == 0 or ids.numel() % n != 0:
        if n == 0:
            return ids.reshape(0, ids.shape[-1] if ids.dim() > 0 else 1).to(torch.int64)
        raise ValueError(f"ids with {ids.numel()} elements do not divide into {n} rows")
    return ids.reshape(n, ids.numel() // n).to(torch.int64).contiguous()


def _cap(softcap) -> float:
    if softcap is None:
        return 0.0
    c = float(softcap)
    if not (c > 0.0 and c != float("inf")):
        raise ValueError("softcap must be finite and positive")
    return c


class _Logprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, ignore_index, cap):
        rows = _as_rows(logits)
        ids2 = _ids_rows(ids, _nrows(rows))
        logp, stats = vls_logp_fwd(rows, ids2, ignore_index, cap)
        ctx.save_for_backward(rows, ids2, stats)
        ctx.meta = (ignore_index, cap, logits.shape)
        return logp.reshape(ids.shape)

    @staticmethod
    def backward(ctx, grad):
        rows, ids2, stats = ctx.saved_tensors
        ignore_index, cap, shape = ctx.meta
        g = grad.reshape(ids2.shape).to(torch.float32).contiguous()
        d = vls_logp_bwd(rows, ids2, g, stats, ignore_index, cap)
        return d.reshape(shape), None, None, None


class _Entropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, cap):
        rows = _as_rows(logits)
        H, stats = vls_entropy_fwd(rows, cap)
        ctx.save_for_backward(rows, H, stats)
        ctx.meta = (cap, logits.shape)
        return H.reshape(logits.shape[:-1])

    @staticmethod
    def backward(ctx, grad):
        rows, H, stats = ctx.saved_tensors
        cap, shape = ctx.meta
        g = grad.reshape(-1).to(torch.float32).contiguous()
        return vls_entropy_bwd(rows, g, H, stats, cap).reshape(shape), None


class _KL(torch.autograd.Function):
    @staticmethod
    def forward(ctx, policy, reference, direction, cap):
        a, b = _as_rows(policy), _as_rows(reference.detach())
        kl, sa, sb = vls_kl_fwd(a, b, direction, cap)
        ctx.save_for_backward(a, b, kl, sa, sb)
        ctx.meta = (direction, cap, policy.shape)
        return kl.reshape(policy.shape[:-1])

    @staticmethod
    def backward(ctx, grad):
        a, b, kl, sa, sb = ctx.saved_tensors
        direction, cap, shape = ctx.meta
        g = grad.reshape(-1).to(torch.float32).contiguous()
        return vls_kl_bwd(a, b, g, kl, sa, sb, direction, cap).reshape(shape), None, None, None


class _Softcap(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, cap):
        xc = x.contiguous()
        ctx.save_for_backward(xc)
        ctx.cap = cap
        return vls_softcap_fwd(xc, cap)

    @staticmethod
    def backward(ctx, gy):
        (xc,) = ctx.saved_tensors
        if gy.dtype not in (torch.float32, xc.dtype):
            gy = gy.to(torch.float32)
        return vls_softcap_bwd(xc, gy.contiguous(), ctx.cap), None


class _Stats(torch.autograd.Function):
    @staticmethod
    def forward(ctx, policy, reference, ids, direction, ignore_index, cap):
        a = _as_rows(policy)
        b = _as_rows(reference.detach()) if reference is not None else None
        ids2 = None
        if ids is not None:
            ids2 = _ids_rows(ids, _nrows(a))
        out = vls_fused_fwd(a, b, ids2, logp=ids is not None, entropy=True, direction=direction,
                            ignore_index=ignore_index, cap=cap)
        ctx.save_for_backward(a, b, ids2, out["stats_a"], out.get("stats_b"), out["H"], out.get("kl"))
        ctx.meta = (direction, ignore_index, cap, policy.shape, ids.shape if ids is not None else None)
        lead = policy.shape[:-1]
        empty = a.new_empty(0, dtype=torch.float32)
        logp = out["logp"].reshape(ids.shape) if ids is not None else empty
        klv = out["kl"].reshape(lead) if b is not None else empty
        return logp, out["H"].reshape(lead), klv

    @staticmethod
    def backward(ctx, g_logp, g_H, g_kl):
        a, b, ids2, sa, sb, H, kl = ctx.saved_tensors
        direction, ignore_index, cap, shape, ids_shape = ctx.meta
        f32 = lambda g, shp: None if g is None else g.reshape(shp).to(torch.float32).contiguous()  # noqa: E731
        gl = f32(g_logp, ids2.shape) if ids2 is not None else None
        gh = f32(g_H, (-1,))
        gk = f32(g_kl, (-1,)) if b is not None else None
        if gl is None and gh is None and gk is None:
            return None, None, None, None, None, None
        fwd = {"stats_a": sa, "stats_b": sb, "H": H, "kl": kl}
        da = vls_fused_bwd(a, fwd, b, ids2, g_logp=gl, g_H=gh, g_kl=gk, direction=direction,
                           ignore_index=ignore_index, cap=cap)
        return da.reshape(shape), None, None, None, None, None


def stats(policy: torch.Tensor, ids: torch.Tensor | None = None, reference: torch.Tensor | None = None,
          direction: str = "reverse", ignore_index: int = -100, softcap: float | None = None):
    """(logp, entropy, kl) of softmax(softcap(policy)) from one read of the
    policy (and one of the reference): logp like ``logprobs`` (empty without
    ids), entropy per row, KL against the detached reference (empty without
    one).  The backward of any weighted sum of the three is one pass."""
    if direction not in ("reverse", "forward"):
        raise ValueError("direction must be 'reverse' or 'forward'")
    return _Stats.apply(policy, reference, ids, direction, int(ignore_index), _cap(softcap))


def logprobs(logits: torch.Tensor, ids: torch.Tensor, ignore_index: int = -100,
             softcap: float | None = None) -> torch.Tensor:
    """log_softmax(softcap(logits))[..., ids]: fp32, shaped like ``ids`` ([..., k] or [...]).

    Ids equal to ``ignore_index`` or outside [0, V) give 0 and no gradient.
    """
    return _Logprobs.apply(logits, ids, int(ignore_index), _cap(softcap))


def entropy(logits: torch.Tensor, softcap: float | None = None) -> torch.Tensor:
    """Entropy of softmax(softcap(logits)) per row (fp32, shape logits.shape[:-1])."""
    return _Entropy.apply(logits, _cap(softcap))


def kl(policy: torch.Tensor, reference: torch.Tensor, direction: str = "reverse",
       softcap: float | None = None) -> torch.Tensor:
    """Per-row KL between softmax(policy) and softmax(reference).

    ``direction="reverse"``: KL(p_policy || p_reference); ``"forward"``:
    KL(p_reference || p_policy).  The gradient flows to ``policy`` only.
    """
    if direction not in ("reverse", "forward"):
        raise ValueError("direction must be 'reverse' or 'forward'")
    return _KL.apply(policy, reference, direction, _cap(softcap))


def softcap(x: torch.Tensor, cap: float = 30.0) -> torch.Tensor:
    """cap * tanh(x / cap), elementwise, in x's dtype."""
    return _Softcap.apply(x, _cap(cap))


class _LinearLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, ids, ignore_index, check):
        h = hidden.reshape(-1, hidden.shape[-1])
        if h.shape[-1] > 1 and h.stride(-1) != 1:
            h = h.contiguous()
        w = weight if weight.stride(-1) == 1 else weight.contiguous()
        ids2 = _ids_rows(ids, h.shape[0])
        logp, st, _ = vls_linear_logp_fwd(h, w, ids2, ignore_index, check=check)
        ctx.save_for_backward(h, w, ids2, st)
        ctx.meta = (ignore_index, hidden.shape, check)
        return logp.reshape(ids.shape)

    @staticmethod
    def backward(ctx, grad):
        h, w, ids2, st = ctx.saved_tensors
        ignore_index, shape, check = ctx.meta
        g = grad.reshape(ids2.shape).to(torch.float32).contiguous()
        dh, dw, _ = vls_linear_logp_bwd(h, w, ids2, g, st, ignore_index, check=check)
        return dh.reshape(shape), dw, None, None, None


def linear_logprobs(hidden: torch.Tensor, weight: torch.Tensor, ids: torch.Tensor,
                    ignore_index: int = -100, check: bool = True) -> torch.Tensor:
    """log_softmax(hidden @ weight^T)[..., ids] without storing the logits.

    hidden: [..., D] and weight: [V, D], both bfloat16 or both float16; ids
    shaped like hidden's leading dims ([...] or [..., k], k <= 16).  The
    gradient flows to hidden and weight.

    Every wait inside the tensor-core kernels is bounded; one that runs out
    makes the kernel return early with invalid outputs and sets a status
    word.  With check=True (the default) the forward and the backward each
    synchronise the device after their kernels, read that word and raise
    VlsDeviceError when it is set.  check=False skips the synchronisation
    (the calls stay asynchronous); ``check_device_error()`` then reports
    the same failures later, for any number of calls at once.
    """
    return _LinearLogprobs.apply(hidden, weight, ids, int(ignore_index), bool(check))


# ---------------------------------------------------------------------------
# training losses
# ---------------------------------------------------------------------------

def _const(t, shape, what: str):
    """A constant input of a loss, of the given shape: float32, contiguous,
    flattened and detached (None stays None).  Dimensions of size 1 and one
    flattened dimension leave no doubt about the order; other shapes are refused."""
    if t is None:
        return None
    have, want = ([d for d in s if d != 1] for s in (t.shape, shape))
    if t.numel() != shape.numel() or (have != want and min(len(have), len(want)) > 1):
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.detach().reshape(-1).to(torch.float32).contiguous()


def _loss_ids(ids: torch.Tensor, logits: torch.Tensor, n: int, k: int | None) -> torch.Tensor:
    """ids shaped like the logits' leading dims (k None), or those and a trailing k."""
    want = logits.shape[:-1] if k is None else (*logits.shape[:-1], k)
    if tuple(ids.shape) != tuple(want):
        raise ValueError(f"ids must have shape {tuple(want)}, not {tuple(ids.shape)}")
    if ids.is_floating_point() or ids.is_complex() or ids.dtype == torch.bool:
        raise TypeError(f"ids must be integers, not {ids.dtype}")
    return ids.detach().reshape(n, k or 1).to(torch.int64).contiguous()


def _mean_weights(ids: torch.Tensor, v: int, ignore_index: int) -> torch.Tensor:
    """[N] weights of the mean over the rows that have a valid id."""
    valid = ((ids != ignore_index) & (ids >= 0) & (ids < v)).any(1).to(torch.float32)
    return valid / valid.sum().clamp(min=1.0)


class _Loss(torch.autograd.Function):
    """loss = call(rows, grad) with the gradient of the logits made by the same
    call.  The backward hands that gradient out (the kernel leaves it alone
    when the upstream gradient is 1 and otherwise makes it again in place with
    the upstream factor, so that it is rounded once); a further backward of a
    retained graph makes it again from the saved statistics."""

    @staticmethod
    def forward(ctx, logits, call, ids, keys, ignore_index, cap, temperature, want):
        rows = _as_rows(logits)
        out = call(rows, want)
        if want:
            ctx.save_for_backward(rows, ids, out["coef"], out["stats"])
            ctx.grad = out["dlogits"]
            ctx.meta = (ignore_index, cap, temperature, logits.shape)
        terms = tuple(out[key] for key in keys)
        ctx.mark_non_differentiable(*terms)
        return (out["loss"], *terms)

    @staticmethod
    @once_differentiable
    def backward(ctx, g, *unused):
        rows, ids, coef, stats = ctx.saved_tensors
        ignore_index, cap, temperature, shape = ctx.meta
        d, ctx.grad = ctx.grad, None
        d = vls_loss_bwd(rows, ids, coef, stats, g.to(torch.float32).contiguous(), ignore_index=ignore_index, cap=cap,
                         temperature=temperature, unless_one=d is not None, dlogits=d)
        return (d.reshape(shape),) + (None,) * 7


def _wants_grad(logits: torch.Tensor) -> bool:
    return torch.is_grad_enabled() and logits.requires_grad


def policy_loss(logits: torch.Tensor, ids: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *,
                ref_logp: torch.Tensor | None = None, weights: torch.Tensor | None = None, clip_low: float = 0.2,
                clip_high: float = 0.2, dual_clip: float | None = None, kl_coef: float = 0.0,
                ignore_index: int = -100, temperature: float = 1.0, softcap: float | None = None):
    """Clipped policy loss with a KL term: (loss, row_loss, logp).

    logits [..., V], ids and the per-token old_logp, advantages, ref_logp and
    weights [...].  Per token, with r = exp(logp - old_logp):
    row_loss = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A), at most
    -dual_clip A for A < 0, plus kl_coef (exp(d) - d - 1), d = ref_logp - logp.
    loss = sum(weights * row_loss); weights default to the mean over the tokens
    whose id is valid.  The gradient flows from ``loss`` to ``logits`` only;
    ``row_loss`` and ``logp`` (0 at ignored ids) are for metrics.
    """
    n, lead = logits.shape[:-1].numel(), logits.shape[:-1]
    ids2 = _loss_ids(ids, logits, n, None)
    cap = _cap(softcap)
    w = _const(weights, lead, "weights") if weights is not None else _mean_weights(ids2, logits.shape[-1], ignore_index)
    old, adv = _const(old_logp, lead, "old_logp"), _const(advantages, lead, "advantages")
    ref = _const(ref_logp, lead, "ref_logp")

    def call(rows, grad):
        return vls_policy_loss(rows, ids2, old, adv, w, ref, clip_low=clip_low, clip_high=clip_high,
                               dual_clip=dual_clip or 0.0, kl_coef=kl_coef, ignore_index=int(ignore_index), cap=cap,
                               temperature=temperature, grad=grad)

    loss, row_loss, logp = _Loss.apply(logits, call, ids2, ("row_loss", "logp"), int(ignore_index), cap, temperature,
                                       _wants_grad(logits))
    return loss, row_loss.reshape(lead), logp.reshape(lead)


def distill_loss(logits: torch.Tensor, ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                 teacher_lse: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                 temperature: float = 1.0, ignore_index: int = -100, softcap: float | None = None):
    """Forward KL from a teacher known by its logits at k ids per row:
    (loss, row_loss).

    logits [..., V]; ids and teacher_logits [..., k]; rows with fewer entries
    are padded with ignore_index.  row_loss = sum_j p_j (log p_j - log q[ids_j])
    with q = softmax(logits / temperature) and p the softmax of teacher_logits /
    temperature over the row's entries, or, with teacher_lse [...] (the
    log-sum-exp of all the teacher's logits / temperature), its true
    probabilities.  loss = sum(weights * row_loss); weights default to the mean
    over the rows with an entry.  The gradient flows from ``loss`` to
    ``logits`` only.
    """
    n, lead = logits.shape[:-1].numel(), logits.shape[:-1]
    if ids.dim() != logits.dim() or ids.shape[-1] < 1:
        raise ValueError(f"ids must have shape {(*lead, 'k')}, not {tuple(ids.shape)}")
    ids2 = _loss_ids(ids, logits, n, ids.shape[-1])
    if tuple(teacher_logits.shape) != tuple(ids.shape):
        raise ValueError(f"teacher_logits must have the ids' shape {tuple(ids.shape)}, not {tuple(teacher_logits.shape)}")
    teacher = teacher_logits.detach().contiguous()
    cap = _cap(softcap)
    w = (_const(weights, lead, "weights") if weights is not None
         else _mean_weights(ids2, logits.shape[-1], ignore_index))
    lse = _const(teacher_lse, lead, "teacher_lse")

    def call(rows, grad):
        return vls_distill_loss(rows, ids2, teacher, w, lse, ignore_index=int(ignore_index), cap=cap,
                                temperature=temperature, grad=grad)

    loss, row_loss = _Loss.apply(logits, call, ids2, ("row_loss",), int(ignore_index), cap, temperature,
                                 _wants_grad(logits))
    return loss, row_loss.reshape(lead)


def preference_loss(logits: torch.Tensor, ids: torch.Tensor, offsets: torch.Tensor | None = None, *,
                    ref_logp: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                    margin: torch.Tensor | None = None, kind: str = "sigmoid", beta: float = 0.1,
                    label_smoothing: float = 0.0, length_average: bool = False, ignore_index: int = -100,
                    softcap: float | None = None):
    """Preference loss of paired sequences: (loss, pair_loss, reward, logp).

    Padded: logits [2P, T, V], ids [2P, T] (ignore_index at prompt and padding
    positions).  Packed: logits [N, V], ids [N] and offsets, int64 [2P + 1] on
    the device, sequence s being rows offsets[s] to offsets[s + 1] - 1.
    Sequence i < P is preferred over sequence P + i.  With R_s the sum (or with
    length_average the mean) of logp - ref_logp over a sequence's valid tokens,
    u = beta (R_i - R_{P+i}) - margin_i and pair_loss is, by ``kind``,
    "sigmoid" -log sigmoid(u) (with label_smoothing, which the others ignore),
    "hinge" max(0, 1 - u) or "squared" (u / beta - 1 / (2 beta))^2.
    loss = sum(weights * pair_loss), weights defaulting to 1/P; reward = beta R.
    The gradient flows from ``loss`` to ``logits`` only.
    """
    n, lead = logits.shape[:-1].numel(), logits.shape[:-1]
    ids2 = _loss_ids(ids, logits, n, None)
    if offsets is None:
        if logits.dim() != 3 or logits.shape[0] % 2 != 0:
            raise ValueError("without offsets, logits must be [2P, T, V]")
        s, t = logits.shape[:2]
        offsets = torch.arange(s + 1, dtype=torch.int64, device=logits.device) * t
    else:
        offsets = offsets.detach().to(torch.int64).contiguous()
    pairs = offsets.numel() // 2
    if pairs < 1 or offsets.numel() != 2 * pairs + 1:
        raise ValueError("offsets must have 2P + 1 elements, P >= 1")
    cap = _cap(softcap)
    per_pair = torch.Size((pairs,))
    w = (_const(weights, per_pair, "weights") if weights is not None
         else torch.full((pairs,), 1.0 / pairs, dtype=torch.float32, device=logits.device))
    ref, mar = _const(ref_logp, lead, "ref_logp"), _const(margin, per_pair, "margin")

    def call(rows, grad):
        return vls_preference_loss(rows, ids2, offsets, ref, w, mar, kind=kind, beta=beta,
                                   label_smoothing=label_smoothing, length_average=length_average,
                                   ignore_index=int(ignore_index), cap=cap, grad=grad)

    loss, pair_loss, reward, logp = _Loss.apply(logits, call, ids2, ("pair_loss", "reward", "logp"), int(ignore_index),
                                                cap, 1.0, _wants_grad(logits))
    return loss, pair_loss, reward, logp.reshape(lead)
