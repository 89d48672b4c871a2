"""Measured cases of the training losses over a vocabulary: the clipped
policy loss with a KL term, the distillation loss from a teacher's top logits
and the preference loss of paired sequences, each with its gradient with
respect to the logits.

``run`` computes a case in plain torch operations (fp32, fp64 where a long sum
needs it) or, with ``own`` set, through the library's binding.  ``exact``
computes the same outputs in fp64 from the definitions, the gradients by
automatic differentiation.
"""

from __future__ import annotations

import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}

# Policy loss.  b sequences of t response tokens; `prompt` is the share of rows
# without a target (prompt and padding tokens of a batch), `shift` reads
# logits[:, :-1] of a [b, t + 1, v] tensor in place, as a causal model's
# training step does.
_POLICY = dict(op="policy", dtype="bf16", prompt=0.0, shift=False, ref=True, clip_low=0.2, clip_high=0.2, dual=0.0,
               cap=0.0, temperature=1.0)
# Distillation.  n rows against a teacher's k top logits; `lse`: the teacher's
# log-sum-exp comes with them (its true probabilities), else they are
# renormalised over the k.
_DISTILL = dict(op="distill", dtype="bf16", cap=0.0, temperature=1.0, lse=False, ignored=0.0)
# Preference.  2 * pairs sequences packed row after row, of lengths spread
# between `short` and `long` tokens, `prompt` the share of rows without a target.
_PREFERENCE = dict(op="preference", dtype="bf16", prompt=0.0, kind="sigmoid", smoothing=0.0, average=False, cap=0.0)


def listed():
    return [
        # one short answer on a small vocabulary: the latency of a call
        dict(_POLICY, name="policy_8x32000", b=1, t=8, v=32000),
        # a training batch at the benchmark's vocabulary: 16 sequences of 512
        # positions, a quarter of them prompt, shifted in place
        dict(_POLICY, name="policy_8192x151936", b=16, t=512, v=151936, prompt=0.25, shift=True, clip_high=0.28),
        # an odd vocabulary, so that rows start at every 2-byte offset; fp16
        dict(_POLICY, name="policy_2747x30011_fp16", b=41, t=67, v=30011, dtype="fp16", prompt=0.1, dual=3.0,
             temperature=0.8),
        # a wide vocabulary behind a final-logit softcap
        dict(_POLICY, name="policy_2048x262144_cap", b=4, t=512, v=262144, cap=30.0, ref=False),
        # a few tokens of a student against 20 logged teacher logits
        dict(_DISTILL, name="distill_16x151936_k20", n=16, v=151936, k=20),
        # a distillation batch, softened by a temperature
        dict(_DISTILL, name="distill_8192x151936_k64", n=8192, v=151936, k=64, temperature=2.0),
        # an odd vocabulary in fp32 against the teacher's true probabilities
        dict(_DISTILL, name="distill_1021x65537_k256_fp32", n=1021, v=65537, k=256, dtype="fp32", lse=True, ignored=0.1),
        # a wide vocabulary, few teacher entries
        dict(_DISTILL, name="distill_2048x262144_k8", n=2048, v=262144, k=8, ignored=0.05),
        # one pair of short answers: the latency of a call
        dict(_PREFERENCE, name="preference_1pair_32000", pairs=1, short=24, long=40, v=32000),
        # a batch of pairs at the benchmark's vocabulary, a third of it prompt
        dict(_PREFERENCE, name="preference_8pairs_151936", pairs=8, short=300, long=700, v=151936, prompt=0.33),
        # many ragged pairs on an odd vocabulary, smoothed labels
        dict(_PREFERENCE, name="preference_29pairs_30011_fp16", pairs=29, short=1, long=111, v=30011, dtype="fp16",
             smoothing=0.1, prompt=0.1),
        # one pair of long answers on a tensor-parallel shard's width, averaged over their lengths
        dict(_PREFERENCE, name="preference_1pair_long_75968", pairs=1, short=3900, long=4300, v=75968, average=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    v = rng.choice([32000, 75968, 151936, 262144]) if rng.random() < 0.4 else _log_uniform(rng, 20000, 262144)
    rows = _log_uniform(rng, 4, min(8192, 8192 * 151936 * 2 // (v * BYTES[dtype])))
    cap = rng.choice([0.0, 0.0, 0.0, 30.0])
    op = rng.choice(["policy", "distill", "preference"])
    if op == "policy":
        b = rng.randint(1, min(16, rows))
        return dict(_POLICY, dtype=dtype, v=v, b=b, t=max(1, rows // b), prompt=rng.choice([0.0, 0.1, 0.3]),
                    shift=rng.random() < 0.3, ref=rng.random() < 0.6, clip_high=rng.choice([0.2, 0.28]),
                    dual=rng.choice([0.0, 3.0]), cap=cap, temperature=rng.choice([1.0, 1.0, 0.7]))
    if op == "distill":
        return dict(_DISTILL, dtype=dtype, v=v, n=rows, k=_log_uniform(rng, 1, 256), cap=cap,
                    temperature=rng.choice([1.0, 2.0]), lse=rng.random() < 0.5, ignored=rng.choice([0.0, 0.1]))
    pairs = rng.randint(1, max(1, min(32, rows // 4)))
    mean = max(2, rows // (2 * pairs))
    return dict(_PREFERENCE, dtype=dtype, v=v, pairs=pairs, short=max(1, mean // 2), long=mean + mean // 2 - 1,
                prompt=rng.choice([0.0, 0.2]), kind=rng.choice(["sigmoid", "sigmoid", "squared"]),
                smoothing=rng.choice([0.0, 0.1]), average=mean > 400 or rng.random() < 0.3, cap=cap)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Lengths of the 2 * pairs sequences, spread over [short, long]."""
    s, span = 2 * case["pairs"], case["long"] - case["short"]
    return [case["short"] + (span * ((7 * i + 3) % s)) // max(1, s - 1) for i in range(s)]


def _rows(case):
    if case["op"] == "policy":
        return case["b"] * case["t"]
    return case["n"] if case["op"] == "distill" else sum(_lengths(case))


def _ignored(case, n):
    return int(n * case["ignored" if case["op"] == "distill" else "prompt"])


def _zipf_logits(shape, gen):
    """Logits whose softmax falls off like a power law over the vocabulary, as
    a language model's does (scaled Gumbel draws)."""
    x = torch.empty(shape, dtype=torch.float32, device="cuda").exponential_(generator=gen)
    return x.clamp_(min=1e-30).log_().mul_(-1.5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    n, v, dt = _rows(case), case["v"], DTYPES[case["dtype"]]
    f32 = dict(dtype=torch.float32, device="cuda")
    cap, tau = case["cap"], case.get("temperature", 1.0)
    st = {"case": case}
    if case["op"] == "policy" and case["shift"]:
        base = torch.zeros((case["b"], case["t"] + 1, v), dtype=dt, device="cuda")
        st["logits"] = base[:, :-1]
        block = [(st["logits"][i], i * case["t"], (i + 1) * case["t"]) for i in range(case["b"])]
    else:
        st["logits"] = torch.empty((n, v), dtype=dt, device="cuda")
        block = [(st["logits"][r:r + 512], r, min(n, r + 512)) for r in range(0, n, 512)]
    k = case["k"] if case["op"] == "distill" else 1
    ids = torch.empty((n, k), dtype=torch.int64, device="cuda")
    score = torch.empty((n, k), **f32)
    lse = torch.empty((n,), **f32)
    for part, r0, r1 in block:
        x = _zipf_logits((r1 - r0, v), gen)
        part.copy_(x)
        z = part.float()
        z = (cap * torch.tanh(z / cap) if cap else z) / tau
        if case["op"] == "distill":
            # the teacher: the student's logits, disturbed; its k largest
            z = z * tau + 0.7 * torch.randn(z.shape, generator=gen, **f32)
            top = z.topk(k, dim=1)
            score[r0:r1], ids[r0:r1] = top.values, top.indices
            lse[r0:r1] = torch.logsumexp(z / tau, 1)
        else:
            # tokens sampled from the model itself
            u = torch.empty(z.shape, **f32).exponential_(generator=gen).clamp_(min=1e-30).log_()
            pick = (z - u).argmax(1, keepdim=True)
            ids[r0:r1] = pick
            score[r0:r1] = z.gather(1, pick) - torch.logsumexp(z, 1, keepdim=True)
        del x, z
    off = _ignored(case, n)
    if off:
        ids[torch.randperm(n, generator=gen, device="cuda")[:off]] = IGNORE
    kept = max(1, n - off)
    valid = (ids[:, 0] != IGNORE).float()
    noise = lambda scale: scale * torch.randn((n,), generator=gen, **f32)  # noqa: E731
    if case["op"] == "policy":
        logp, step = score[:, 0], noise(0.15)
        # rounding may not decide on which side of a clip border a token lies
        for edge in (math.log1p(-case["clip_low"]), math.log1p(case["clip_high"])):
            step = torch.where((step - edge).abs() < 2e-3, torch.full_like(step, 0.9 * edge), step)
        adv = torch.randn((case["b"], 1), generator=gen, **f32).expand(case["b"], case["t"]).reshape(n)
        st |= dict(ids=ids[:, 0].clone(), old=logp - step, adv=adv.contiguous(), weights=valid / kept,
                   ref=logp + noise(0.3) if case["ref"] else None)
    elif case["op"] == "distill":
        st |= dict(ids=ids, teacher=score, lse=lse if case["lse"] else None, weights=valid / kept)
    else:
        # the model has drifted from its reference by 0.02 to 0.05 nats a token, up or down over a whole sequence
        offsets = torch.tensor([0] + _lengths(case), dtype=torch.int64).cumsum(0).cuda()
        drift = (0.02 + 0.03 * torch.rand((2 * case["pairs"],), generator=gen, **f32))
        drift *= 1.0 - 2.0 * torch.randint(0, 2, drift.shape, generator=gen, device="cuda")
        drift = torch.repeat_interleave(drift, offsets.diff(), output_size=n)
        st |= dict(ids=ids[:, 0].clone(), ref=score[:, 0] - drift + noise(0.1), offsets=offsets,
                   weights=torch.full((case["pairs"],), 1.0 / case["pairs"], **f32))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_logits(x, cap, tau):
    """(z [n, v] fp32 after cap and temperature, dz/dx or 1/tau)."""
    x = x.reshape(-1, x.shape[-1]).float()
    if not cap:
        return x / tau, 1.0 / tau
    th = torch.tanh(x / cap)
    return th * (cap / tau), (1.0 - th * th) / tau


def _plain_softmax(z):
    """(exp(z - m), its row sums, m)."""
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    return e, e.sum(1, keepdim=True), m


def _plain_logp(z, s, m, ids):
    return z.gather(1, ids.clamp(min=0)) - m - torch.log(s)


def _plain_grad(e, s, slope, ids, valid, coef, dtype):
    """sum_j coef_j (onehot_j - softmax), times dz/dx, in the logits' dtype."""
    d = e * (-coef.sum(1, keepdim=True) / s)
    d.scatter_add_(1, torch.where(valid, ids, torch.zeros_like(ids)), coef)
    return (d * slope).to(dtype)


def _plain_policy(st):
    c, ids = st["case"], st["ids"].reshape(-1, 1)
    z, slope = _plain_logits(st["logits"], c["cap"], c["temperature"])
    e, s, m = _plain_softmax(z)
    valid = ids != IGNORE
    logp = torch.where(valid, _plain_logp(z, s, m, ids), 0.0)[:, 0]
    on, adv, w = valid[:, 0], st["adv"], st["weights"]
    ratio = torch.exp(logp - st["old"])
    clipped = ratio.clamp(1.0 - c["clip_low"], 1.0 + c["clip_high"])
    gain = torch.minimum(ratio * adv, clipped * adv)
    through = (clipped == ratio) | (ratio * adv < clipped * adv)
    if c["dual"]:
        floor = c["dual"] * adv
        through = through & ((adv >= 0) | (gain > floor))
        gain = torch.where(adv < 0, torch.maximum(gain, floor), gain)
    row, dlogp = -gain, torch.where(through, -ratio * adv, 0.0)
    if st["ref"] is not None:
        far = st["ref"] - logp
        row = row + 0.04 * (torch.expm1(far) - far)
        dlogp = dlogp - 0.04 * torch.expm1(far)
    row = torch.where(on, row, 0.0)
    coef = torch.where(on, dlogp * w, 0.0)[:, None]
    return {"loss": (row.double() * w).sum().float(), "row_loss": row, "logp": logp,
            "dlogits": _plain_grad(e, s, slope, ids, valid, coef, st["logits"].dtype)}


def _plain_distill(st):
    c, ids = st["case"], st["ids"]
    tau, w = c["temperature"], st["weights"]
    z, slope = _plain_logits(st["logits"], c["cap"], tau)
    e, s, m = _plain_softmax(z)
    valid = ids != IGNORE
    logq = _plain_logp(z, s, m, ids)
    t = torch.where(valid, st["teacher"] / tau, -torch.inf)
    if st["lse"] is not None:
        logt = t - st["lse"][:, None]
    else:
        te, ts, tm = _plain_softmax(torch.where(valid.any(1, keepdim=True), t, 0.0))
        logt = t - tm - torch.log(ts)
    p = torch.exp(logt)
    row = torch.where(p > 0, p * (logt - logq), 0.0).sum(1)
    coef = torch.where(valid, -p * w[:, None], 0.0)
    return {"loss": (row.double() * w).sum().float(), "row_loss": row,
            "dlogits": _plain_grad(e, s, slope, ids, valid, coef, st["logits"].dtype)}


def _plain_preference(st):
    c, ids, w = st["case"], st["ids"].reshape(-1, 1), st["weights"]
    z, slope = _plain_logits(st["logits"], c["cap"], 1.0)
    e, s, m = _plain_softmax(z)
    valid = ids != IGNORE
    logp = torch.where(valid, _plain_logp(z, s, m, ids), 0.0)[:, 0]
    pairs, off = c["pairs"], st["offsets"]
    seq = torch.bucketize(torch.arange(logp.numel(), device=off.device), off, right=True) - 1
    on = valid[:, 0]
    total = torch.zeros(2 * pairs, dtype=torch.float64, device=off.device)
    total = total.index_add(0, seq, torch.where(on, logp.double() - st["ref"].double(), 0.0))
    scale = torch.ones_like(total)
    if c["average"]:
        scale = 1.0 / torch.zeros_like(total).index_add(0, seq, on.double()).clamp(min=1.0)
    total = total * scale
    u = 0.1 * (total[:pairs] - total[pairs:])
    if c["kind"] == "sigmoid":
        lam = c["smoothing"]
        soft = lambda x: x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731  log(1 + e^x)
        pair = (1 - lam) * soft(-u) + lam * soft(u)
        du = -(1 - lam) / (1 + torch.exp(u)) + lam / (1 + torch.exp(-u))
    else:  # squared distance of the paired log ratio from 1 / (2 beta)
        pair = (u / 0.1 - 5.0) ** 2
        du = 2.0 * (u / 0.1 - 5.0) / 0.1
    g = 0.1 * du * w
    g = torch.cat([g, -g]) * scale
    coef = torch.where(on, g[seq], 0.0).float()[:, None]
    return {"loss": (pair * w).sum().float(), "pair_loss": pair.float(), "reward": (0.1 * total).float(), "logp": logp,
            "dlogits": _plain_grad(e, s, slope, ids, valid, coef, st["logits"].dtype)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    c = st["case"]
    if not own:
        return {"policy": _plain_policy, "distill": _plain_distill, "preference": _plain_preference}[c["op"]](st)
    from vocab_log_softmax_gb300 import binding as B

    if c["op"] == "policy":
        o = B.vls_policy_loss(st["logits"], st["ids"], st["old"], st["adv"], st["weights"], st["ref"],
                              clip_low=c["clip_low"], clip_high=c["clip_high"], dual_clip=c["dual"],
                              kl_coef=0.04 if c["ref"] else 0.0, cap=c["cap"], temperature=c["temperature"])
        return {key: o[key] for key in ("loss", "row_loss", "logp", "dlogits")}
    if c["op"] == "distill":
        o = B.vls_distill_loss(st["logits"], st["ids"], st["teacher"], st["weights"], st["lse"], cap=c["cap"],
                               temperature=c["temperature"])
        return {key: o[key] for key in ("loss", "row_loss", "dlogits")}
    o = B.vls_preference_loss(st["logits"], st["ids"], st["offsets"], st["ref"], st["weights"], kind=c["kind"], beta=0.1,
                              label_smoothing=c["smoothing"], length_average=c["average"], cap=c["cap"])
    return {key: o[key] for key in ("loss", "pair_loss", "reward", "logp", "dlogits")}


def work(case):
    """Rows with a target are read once; every gradient row is written once
    (the preference loss reads its rows a second time: a row's gradient needs
    the sums over its whole pair).  About 5 operations an element read for the
    softmax sums and 5 for the gradient."""
    n, v = _rows(case), case["v"]
    kept = n - _ignored(case, n)
    reads = 2 if case["op"] == "preference" else 1
    small = {"policy": 28, "distill": 12 * case.get("k", 1) + 12, "preference": 20}[case["op"]]
    return {"bytes": (reads * kept + n) * v * BYTES[case["dtype"]] + n * small, "flops": 10 * kept * v}


# ---------------------------------------------------------------------------
# the definitions in fp64
# ---------------------------------------------------------------------------

def _exact_policy(c, st, logp, on):
    adv, w = st["adv"].double(), st["weights"].double()
    ratio = torch.exp(logp - st["old"].double())
    gain = torch.minimum(ratio * adv, ratio.clamp(1 - c["clip_low"], 1 + c["clip_high"]) * adv)
    if c["dual"]:
        gain = torch.where(adv < 0, torch.maximum(gain, c["dual"] * adv), gain)
    row = -gain
    if st["ref"] is not None:
        far = st["ref"].double() - logp
        row = row + 0.04 * (torch.exp(far) - far - 1)
    row = torch.where(on, row, 0.0)
    return (row * w).sum(), {"row_loss": row, "logp": logp}


def _exact_distill(c, st, logq, valid):
    t = (st["teacher"].double() / c["temperature"]).masked_fill(~valid, -torch.inf)
    lse = st["lse"].double() if st["lse"] is not None else torch.logsumexp(t, 1)
    logt = t - torch.where(valid.any(1), lse, 0.0)[:, None]
    p = torch.exp(logt)
    row = torch.where(valid, p * (logt.masked_fill(~valid, 0.0) - logq), 0.0).sum(1)
    return (row * st["weights"].double()).sum(), {"row_loss": row}


def _exact_preference(c, st, logp, on):
    off = st["offsets"].tolist()
    ratio = torch.where(on, logp - st["ref"].double(), 0.0)
    total = []
    for a, b in zip(off[:-1], off[1:]):
        total.append(ratio[a:b].sum() / (max(1, int(on[a:b].sum())) if c["average"] else 1))
    total = torch.stack(total)
    gap = total[:c["pairs"]] - total[c["pairs"]:]
    if c["kind"] == "sigmoid":
        ls = torch.nn.functional.logsigmoid
        pair = -(1 - c["smoothing"]) * ls(0.1 * gap) - c["smoothing"] * ls(-0.1 * gap)
    else:
        pair = (gap - 1 / (2 * 0.1)) ** 2
    return (pair * st["weights"].double()).sum(), {"pair_loss": pair, "reward": 0.1 * total, "logp": logp}


def exact(case, seed):
    """fp64 throughout; the gradient by automatic differentiation, a block of
    rows at a time."""
    st = prepare(case, seed)
    x = st["logits"].reshape(-1, case["v"])
    n, cap, tau = x.shape[0], case["cap"], case.get("temperature", 1.0)
    ids = st["ids"].reshape(n, -1)
    valid = ids != IGNORE
    rows = max(1, (1 << 27) // case["v"])

    def logp_of(r0, z):
        if cap:
            z = cap * torch.tanh(z / cap)
        got = torch.log_softmax(z / tau, 1).gather(1, ids[r0:r0 + z.shape[0]].clamp(min=0))
        return torch.where(valid[r0:r0 + z.shape[0]], got, 0.0)

    with torch.no_grad():
        logp = torch.cat([logp_of(r0, x[r0:r0 + rows].double()) for r0 in range(0, n, rows)])
    with torch.enable_grad():
        leaf = logp.requires_grad_(True)
        one = case["op"] != "distill"
        rule = {"policy": _exact_policy, "distill": _exact_distill, "preference": _exact_preference}[case["op"]]
        loss, out = rule(case, st, leaf[:, 0] if one else leaf, valid[:, 0] if one else valid)
        (g,) = torch.autograd.grad(loss, leaf)
        grad = torch.empty((n, case["v"]), dtype=torch.float64, device="cuda")
        for r0 in range(0, n, rows):
            z = x[r0:r0 + rows].double().requires_grad_(True)
            (grad[r0:r0 + rows],) = torch.autograd.grad(logp_of(r0, z), z, g[r0:r0 + rows])
    return {key: v.detach() for key, v in dict(out, loss=loss, dlogits=grad).items()}
