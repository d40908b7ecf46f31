"""Measured cases of the training step around the projection: token embedding
and its gradient, the clipped policy loss and the preference loss (forward and
backward), and the AdamW step over many tensors.

``own`` chooses between the plain torch form (fp32, or fp64 where a border or a
long sum decides) and the library's kernels; both take what ``prepare`` gives.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
E4M3_MIN = 2.0 ** -9
BLOCK = 128


def listed():
    return [
        # one decoded token's row (latency)
        dict(name="embed_1", op="embed", n=1, vocab=151936, hidden=4096, weight="bf16", scale=1.0, ids="uniform"),
        # a training batch: common tokens, padding, the scale of tied embeddings
        dict(name="embed_16384", op="embed", n=16384, vocab=151936, hidden=4096, weight="bf16", scale=64.0, ids="zipf"),
        # a decode batch's or a prefill's rows out of the 8-bit matrix that the logits use
        dict(name="embed_fp8_777", op="embed", n=777, vocab=128256, hidden=4096, weight="e4m3", scale=1.0, ids="zipf"),
        # the whole gradient of a training batch, every untouched row zero
        dict(name="embed_grad_16384", op="embed_grad", n=16384, vocab=151936, hidden=4096, into="bf16", scale=1.0,
             ids="zipf"),
        # a micro-batch added to the fp32 accumulator that the projection's backward fills
        dict(name="embed_grad_acc_4096", op="embed_grad", n=4096, vocab=151936, hidden=4096, into="fp32_acc",
             scale=64.0, ids="zipf"),
        # a micro-batch of a few answers: sequence means, one advantage per answer
        dict(name="policy_512", op="policy", n=512, sequences=7, advantage="sequence", reduction="sequence_mean",
             ref=True, kl="k3", dual_clip=0.0),
        # the rollouts of a whole step, clipped twice, KL to the reference
        dict(name="policy_1048576", op="policy", n=1048576, sequences=256, advantage="token", reduction="mean",
             ref=True, kl="k3", dual_clip=3.0),
        # a few pairs
        dict(name="preference_4", op="preference", n=2500, pairs=4, kind="sigmoid", ref=True, average=False),
        # a batch of pairs over long answers, lengths normalised
        dict(name="preference_512", op="preference", n=1000001, pairs=512, kind="sigmoid", ref=True, average=True),
        # the norm weights of a model: many small tensors (latency)
        dict(name="adamw_129x4096", op="adamw", tensors=129, base=4096, ragged=False, param="bf16", grad="bf16",
             state="fp32", copy=False, step=1000, beta2=0.95),
        # a vocabulary matrix with its fp32 gradient accumulator, fp32 states
        dict(name="adamw_vocab", op="adamw", tensors=1, base=128256 * 4096, ragged=False, param="bf16", grad="fp32",
             state="fp32", copy=False, step=1000, beta2=0.95),
        # the same in 8-bit states with a bf16 gradient
        dict(name="adamw_vocab_8bit", op="adamw", tensors=1, base=151936 * 4096, ragged=False, param="bf16",
             grad="bf16", state="e4m3", copy=False, step=1000, beta2=0.999),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "policy", "policy", "preference", "adamw", "adamw"])
    if op in ("embed", "embed_grad"):
        weight = rng.choice(["bf16", "bf16", "fp32", "e4m3"])
        step = 128 if op == "embed" and weight == "e4m3" else 64
        hidden = step * _log_int(rng, 2, 4096 // step)
        c = dict(op=op, n=_log_int(rng, 1, 32768), vocab=_log_int(rng, 1000, 128256), hidden=hidden,
                 scale=rng.choice([1.0, round(hidden ** 0.5, 3)]), ids=rng.choice(["zipf", "uniform", "one"]))
        if op == "embed":
            c["weight"] = weight
        else:
            c["into"] = rng.choice(["bf16", "fp32", "bf16_acc", "fp32_acc"])
        return c
    if op == "policy":
        n = _log_int(rng, 1, 1048576)
        reduction = rng.choice(["mean", "sum", "sequence_mean"])
        kl = rng.choice(["k1", "k2", "k3", "none"])
        return dict(op=op, n=n, sequences=_log_int(rng, 1, max(1, min(4096, n // 2))),
                    advantage=rng.choice(["token", "sequence"]), reduction=reduction, ref=kl != "none", kl=kl,
                    dual_clip=rng.choice([0.0, 3.0]))
    if op == "preference":
        n = _log_int(rng, 2, 1000000)
        return dict(op=op, n=n, pairs=_log_int(rng, 1, max(1, min(2048, n // 4))),
                    kind=rng.choice(["sigmoid", "hinge", "squared"]), ref=rng.random() < 0.7,
                    average=rng.random() < 0.5)
    tensors = _log_int(rng, 1, 200)
    return dict(op=op, tensors=tensors, base=_log_int(rng, 100, 2 ** 27 // tensors), ragged=True,
                param=rng.choice(["bf16", "fp32"]), grad=rng.choice(["bf16", "fp32"]),
                state=rng.choice(["fp32", "e4m3"]), copy=rng.random() < 0.3, step=_log_int(rng, 1, 100000),
                beta2=rng.choice([0.95, 0.999]))


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CLIP_LOW, CLIP_HIGH, KL_WEIGHT = 0.2, 0.28, 0.05
BETA = {"sigmoid": 0.1, "hinge": 0.05, "squared": 0.1}
SMOOTH = 0.1
ADAMW = dict(lr=3e-4, beta1=0.9, eps=1e-8, weight_decay=0.1)


def _sizes(case):
    """Elements of each tensor: all alike, or from a few to 1.6 times base."""
    if not case["ragged"]:
        return [case["base"]] * case["tensors"]
    return [1 + case["base"] * (7 + (i * 7919 + 331) % 1543) // 1000 for i in range(case["tensors"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _ids(case, g):
    n, v = case["n"], case["vocab"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if case["ids"] == "uniform":
        ids = (u * v).long()
    elif case["ids"] == "zipf":
        p = torch.arange(1, v + 1, device="cuda", dtype=torch.float64) ** -1.1
        ids = torch.searchsorted((p.cumsum(0) / p.sum()), u)
    else:   # one token in most places: a filler, or a mask token
        ids = torch.where(u < 0.9, v // 3, (u * v).long())
    ids = ids.clamp(0, v - 1).to(torch.int32)
    if n > 8:   # padding
        ids[torch.rand(n, generator=g, device="cuda") < 0.05] = -100
    return ids


def _bounds(n, sequences, g):
    """int32 [sequences + 1] of packed sequences, some of them empty, over at most n tokens."""
    w = torch.rand(sequences, generator=g, device="cuda", dtype=torch.float64) ** 2
    w[torch.rand(sequences, generator=g, device="cuda") < 0.03] = 0.0
    used = n - (n // 50 if n > 100 else 0)   # the buffer's end holds no sequence
    ends = (w.cumsum(0) / w.sum().clamp(min=1e-30) * used).round().clamp(max=used)
    return torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), ends]).to(torch.int32)


def _token_targets(n, cu, g):
    """int32 [n] as the projection's targets: prompts and one whole sequence are ignored."""
    t = torch.randint(0, 151936, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu.long(), pos, right=True) - 1
    count = cu.shape[0] - 1
    inside = (seq >= 0) & (seq < count)
    s = seq.clamp(0, count - 1)
    start, length = cu.long()[s], cu.long()[s + 1] - cu.long()[s]
    share = torch.rand(count, generator=g, device="cuda") * 0.5
    t[inside & ((pos - start).float() < share[s] * length)] = -100
    if count > 2:
        t[inside & (seq == count // 2)] = -100
    return t


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, v, h = case["n"], case["vocab"], case["hidden"]
        st = dict(case=case, ids=_ids(case, g))
        if op == "embed":
            w = _normal((v, h), g, 0.02)
            if case["weight"] == "e4m3":
                pad = torch.nn.functional.pad(w, (0, 0, 0, -v % BLOCK)).view(-1, BLOCK, h // BLOCK, BLOCK)
                st["ws"] = pad.abs().amax((1, 3)) / E4M3_MAX
                st["w"] = (pad / st["ws"][:, None, :, None]).view(-1, h)[:v].clamp(-E4M3_MAX, E4M3_MAX).to(
                    torch.float8_e4m3fn)
            else:
                st["w"], st["ws"] = w.to(_TYPES[case["weight"]]), None
            return st
        st["dy"] = _normal((n, h), g, 0.01).to(torch.bfloat16)
        if case["into"].endswith("_acc"):
            st["acc"] = _normal((v, h), g, 0.05).to(_TYPES[case["into"][:4]])
        return st
    if op in ("policy", "preference"):
        n = case["n"]
        sequences = case["sequences"] if op == "policy" else 2 * case["pairs"]
        cu = _bounds(n, sequences, g)
        st = dict(case=case, cu=cu, targets=_token_targets(n, cu, g), one=torch.ones(1, device="cuda"))
        off = st["targets"] < 0
        logp = -_normal((n,), g, 1.5).abs()
        ref = torch.minimum(logp + _normal((n,), g, 0.3), torch.zeros_like(logp)) if case["ref"] else None
        st["logp"] = logp.masked_fill(off, 0.0)   # as the log-prob entry leaves ignored rows
        st["ref"] = ref.masked_fill(off, 0.0) if ref is not None else None
        if op == "policy":
            st["old"] = (logp + _normal((n,), g, 0.15)).clamp(max=0.0).masked_fill(off, 0.0)
            st["adv"] = _normal((n if case["advantage"] == "token" else sequences,), g)
        return st
    # the tensors are views of flat buffers, each on a border of blocks; what lies between them is zero
    sizes = _sizes(case)
    starts = [0]
    for size in sizes:
        starts.append(starts[-1] + -(-size // BLOCK) * BLOCK)
    total = starts[-1]
    sigma, live = 0.01, None
    if len(sizes) > 1:
        blocks = torch.tensor([-(-size // BLOCK) for size in sizes], device="cuda")
        each = torch.arange(len(sizes), device="cuda").repeat_interleave(blocks).repeat_interleave(BLOCK)
        sigma = 0.01 * torch.exp(0.5 * torch.sin(each.float()))
        inside = torch.arange(total, device="cuda") - torch.tensor(starts[:-1], device="cuda")[each]
        live = inside < torch.tensor(sizes, device="cuda")[each]
    elif total > sizes[0]:
        live = torch.arange(total, device="cuda") < sizes[0]

    def fresh(std, exp=False):
        x = _normal((total,), g, std)
        x = (x.exp_() if exp else x).mul_(sigma)
        return x if live is None else x.mul_(live)

    st = dict(case=case, p=_normal((total,), g, 0.02), g=fresh(1.0).to(_TYPES[case["grad"]]))
    st["p"] = (st["p"] if live is None else st["p"].mul_(live)).to(_TYPES[case["param"]])
    st["m"], st["v"] = fresh(0.2), fresh(0.3, exp=True)   # v: its root so far
    if case["state"] == "e4m3":
        st["m"], st["ms"] = _to_blocks(st["m"])
        st["v"], st["vs"] = _to_blocks(st["v"])
    else:
        st["v"].square_()
    if case["copy"]:
        st["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
    if own:   # the handle that a program keeps beside its parameters
        import chunked_lm_head_amd as lm
        of = lambda name: [st[name][a:a + k] for a, k in zip(starts, sizes)] if name in st else None  # noqa: E731
        scales = lambda name: [st[name][a // BLOCK:a // BLOCK + -(-k // BLOCK)]  # noqa: E731
                               for a, k in zip(starts, sizes)] if name in st else [None] * len(sizes)
        states = [lm.AdamWState(*t) for t in zip(of("m"), of("v"), scales("ms"), scales("vs"))]
        st["plan"] = lm.adamw_plan(of("p"), of("g"), states, of("copy"))
    return st


# -------------------------------------------------------------- plain forms

def _to_blocks(x):
    """e4m3 values and the scales of blocks of 128 consecutive elements."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    amax = b.abs().amax(1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    q = (b / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(-1)[:n].contiguous(), scale


def _root_blocks(v):
    """The same of sqrt(v), where no non-zero root becomes zero."""
    n = v.numel()
    b = torch.nn.functional.pad(v.sqrt(), (0, -n % BLOCK)).view(-1, BLOCK)
    amax = b.amax(1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    y = (b / scale[:, None]).clamp(max=E4M3_MAX)
    y = torch.where(b > 0, y.clamp(min=E4M3_MIN), 0.0)
    return y.to(torch.float8_e4m3fn).view(-1)[:n].contiguous(), scale


def _of_blocks(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK)[:q.numel()]


def _plain_embed(st):
    c, ids, w = st["case"], st["ids"], st["w"]
    row = ids.clamp(min=0).long()
    y = w[row].float()
    if c["weight"] == "e4m3":
        y = (y.view(y.shape[0], -1, BLOCK) * st["ws"][row // BLOCK][:, :, None]).view(y.shape)
    y = torch.where((ids >= 0)[:, None], y * c["scale"], 0.0)
    return y if c["weight"] == "fp32" else y.to(torch.bfloat16)


def _plain_embed_grad(st):
    c, ids = st["case"], st["ids"]
    live = ids >= 0
    rows = torch.where(live[:, None], st["dy"].float() * c["scale"], 0.0)
    sums = torch.zeros(c["vocab"], c["hidden"], device="cuda").index_add_(0, ids.clamp(min=0).long(), rows)
    if "acc" in st:
        return st["acc"].copy_(st["acc"].float().add_(sums))
    return sums.to(_TYPES[c["into"]])


def _sequence_of(cu, n):
    """Sequence of each token (clamped) and whether it has one."""
    seq = torch.searchsorted(cu, torch.arange(n, device=cu.device, dtype=torch.int32), right=True) - 1
    count = cu.shape[0] - 1
    return seq.clamp(0, count - 1), (seq >= 0) & (seq < count)


def _plain_policy(st):
    c, logp, cu = st["case"], st["logp"], st["cu"]
    n, sequences = logp.shape[0], cu.shape[0] - 1
    seq, inside = _sequence_of(cu, n)
    valid = inside & (st["targets"] >= 0)
    adv = st["adv"] if c["advantage"] == "token" else st["adv"][seq]
    gap = torch.where(valid, logp.double() - st["old"].double(), 0.0)   # the border in 64 bits
    r = gap.float().exp()
    above, below = gap > math.log1p(CLIP_HIGH), gap < math.log1p(-CLIP_LOW)
    up = adv >= 0
    rho = torch.where(up, r.clamp(max=1.0 + CLIP_HIGH), r.clamp(min=1.0 - CLIP_LOW))
    clipped = torch.where(up, above, below)
    if c["dual_clip"]:
        far = ~up & (gap > math.log(c["dual_clip"]))
        rho = torch.where(far, c["dual_clip"], rho)
        clipped = clipped | far
    loss = -adv * rho
    slope = torch.where(clipped, 0.0, -adv * r)
    kl = torch.zeros_like(logp)
    if c["ref"]:
        d = torch.where(valid, logp - st["ref"], 0.0)
        if c["kl"] == "k1":
            kl, dk = d, torch.ones_like(d)
        elif c["kl"] == "k2":
            kl, dk = d.square() / 2, d
        else:
            kl, dk = torch.expm1(-d) + d, -torch.expm1(-d)
        loss = loss + KL_WEIGHT * kl
        slope = slope + KL_WEIGHT * dk
    one = valid.double()
    total = one.sum()
    if c["reduction"] == "sequence_mean":
        per = torch.zeros(sequences, dtype=torch.float64, device="cuda").index_add_(0, seq, one)
        weight = (1.0 / (sequences * per.clamp(min=1.0)))[seq]
    elif c["reduction"] == "mean":
        weight = 1.0 / total.clamp(min=1.0)
    else:
        weight = torch.ones((), dtype=torch.float64, device="cuda")
    out = torch.where(valid, loss.double() * weight, 0.0).sum()
    back = torch.expm1(-gap) + gap
    stats = torch.stack([torch.where(valid, x.double(), 0.0).sum() for x in (kl, clipped, r, back)])
    stats = (stats / total.clamp(min=1.0)).float()
    dlogp = torch.where(valid, slope * weight.float(), 0.0) * st["one"]
    return out.float(), stats, dlogp


def _plain_preference(st):
    c, logp, cu = st["case"], st["logp"], st["cu"]
    n, pairs, beta = logp.shape[0], c["pairs"], BETA[c["kind"]]
    seq, inside = _sequence_of(cu, n)
    valid = inside & (st["targets"] >= 0)
    gain = logp.double() - st["ref"].double() if c["ref"] else logp.double()
    sums = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda")
    s = sums.index_add(0, seq, torch.where(valid, gain, 0.0))
    if c["average"]:
        share = 1.0 / sums.index_add(0, seq, valid.double()).clamp(min=1.0)
    else:
        share = torch.ones_like(sums)
    s = s * share
    h = beta * (s[:pairs] - s[pairs:])
    if c["kind"] == "sigmoid":
        # -log sigmoid(x) = log(1 + e^-x)
        minus = torch.log1p(torch.exp(-h.abs())) + (-h).clamp(min=0)
        plus = minus + h
        each = (1.0 - SMOOTH) * minus + SMOOTH * plus
        slope = torch.sigmoid(h) - (1.0 - SMOOTH)
    elif c["kind"] == "hinge":
        each, slope = (1.0 - h).clamp(min=0), -(h < 1.0).double()
    else:
        each, slope = ((h - 0.5) / beta).square(), 2.0 * (h - 0.5) / beta ** 2
    coef = beta * slope / pairs
    coef = (torch.cat([coef, -coef]) * share).float()
    dlogp = torch.where(valid, coef[seq], 0.0) * st["one"]
    return each.mean().float(), (beta * s).float(), dlogp


def _plain_adamw(st):
    c = st["case"]
    beta1, lr, beta2, t = ADAMW["beta1"], ADAMW["lr"], c["beta2"], c["step"]
    p, g = st["p"].float(), st["g"].float()
    if c["state"] == "e4m3":
        m, v = _of_blocks(st["m"], st["ms"]), _of_blocks(st["v"], st["vs"]).square_()
    else:
        m, v = st["m"], st["v"]
    m = m * beta1 + g * (1.0 - beta1)
    v = v * beta2 + g.square() * (1.0 - beta2)
    root = v.sqrt().mul_(1.0 / math.sqrt(1.0 - beta2 ** t)).add_(ADAMW["eps"])
    p = p * (1.0 - lr * ADAMW["weight_decay"]) - (m / root).mul_(lr / (1.0 - beta1 ** t))
    st["p"].copy_(p)
    if c["copy"]:
        st["copy"].copy_(p)
    if c["state"] == "e4m3":
        for name, scale, (q, s) in (("m", "ms", _to_blocks(m)), ("v", "vs", _root_blocks(v))):
            st[name].copy_(q)
            st[scale].copy_(s)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _adamw_out(st)


def _adamw_out(st):
    return {name: st[name] for name in ("p", "m", "v", "ms", "vs", "copy") if name in st}


# ------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import chunked_lm_head_amd as lm
        if op == "embed":
            return lm.embedding_forward(state["ids"], state["w"], scale=c["scale"], weight_scale=state["ws"])
        if op == "embed_grad":
            if "acc" in state:
                return lm.embedding_backward(state["dy"], state["ids"], c["vocab"], scale=c["scale"], acc=state["acc"])
            return lm.embedding_backward(state["dy"], state["ids"], c["vocab"], scale=c["scale"],
                                         out_dtype=_TYPES[c["into"]])
        if op == "policy":
            how = dict(clip_low=CLIP_LOW, clip_high=CLIP_HIGH, dual_clip=c["dual_clip"],
                       kl_weight=KL_WEIGHT if c["ref"] else 0.0, kl_kind=c["kl"] if c["ref"] else "k3",
                       reduction=c["reduction"])
            given = (state["logp"], state["adv"], state["old"], state["ref"], state["targets"], state["cu"])
            f = lm.policy_loss_forward(*given, **how)
            return f.loss, f.stats, lm.policy_loss_backward(state["one"], f.weights, *given, **how)
        if op == "preference":
            f = lm.preference_loss_forward(state["logp"], state["cu"], state["ref"], state["targets"],
                                           kind=c["kind"], beta=BETA[c["kind"]],
                                           label_smoothing=SMOOTH if c["kind"] == "sigmoid" else 0.0,
                                           average=c["average"])
            return f.loss, f.rewards, lm.preference_loss_backward(state["one"], f.coef, c["n"], state["cu"],
                                                                  state["targets"])
        lm.adamw_step(state["plan"], c["step"], beta2=c["beta2"], **ADAMW)
        return _adamw_out(state)
    return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "policy": _plain_policy,
            "preference": _plain_preference, "adamw": _plain_adamw}[op](state)


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, v, h = case["n"], case["vocab"], case["hidden"]
        # rows that are touched: about n of uniform ids, fewer where some ids are common
        touched = min(v, n) if case["ids"] == "uniform" else min(v, n) // 3 + 1 if case["ids"] == "zipf" else n // 10 + 1
        if op == "embed":
            wb, ob = {"bf16": (2, 2), "fp32": (4, 4), "e4m3": (1, 2)}[case["weight"]]
            return dict(bytes=4 * n + touched * h * wb + n * h * ob, flops=n * h)
        wb = 4 if case["into"].startswith("fp32") else 2
        rows = 2 * touched if case["into"].endswith("_acc") else v
        return dict(bytes=4 * n + 2 * n * h + rows * h * wb, flops=2 * n * h)
    if op == "policy":
        each = 4 * (3 + case["ref"] + (case["advantage"] == "token")) + 4
        return dict(bytes=each * case["n"] + 8 * case["sequences"], flops=40 * case["n"])
    if op == "preference":
        return dict(bytes=(4 * (2 + case["ref"]) + 4) * case["n"] + 24 * case["pairs"], flops=4 * case["n"])
    n = sum(_sizes(case))
    per = 2 * (2 if case["param"] == "bf16" else 4) + (2 if case["grad"] == "bf16" else 4)
    per += (16 if case["state"] == "fp32" else 4 + 16 / BLOCK) + (2 if case["copy"] else 0)
    return dict(bytes=int(per * n), flops=20 * n)


# ------------------------------------------------------ definition, 64 bits

def _e4m3_64(y):
    """Nearest e4m3 value (ties to even) of fp64 values within +-448."""
    mag = y.abs()
    e = torch.floor(torch.log2(torch.where(mag > 0, mag, 1.0))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(y) * torch.clamp(torch.round(mag / step) * step, max=E4M3_MAX)


def _exact_blocks(x, root):
    """Values over their block's scale, and the scales, of 64-bit x."""
    n = x.numel()
    full = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:n] = x
    full = full.view(-1, BLOCK)
    s = full.abs().amax(1) / E4M3_MAX
    s[s == 0] = 1.0
    y = full / s[:, None]
    if root:
        y[(full > 0) & (y < E4M3_MIN)] = E4M3_MIN
    return _e4m3_64(y).view(-1)[:n], s


def _exact_adamw_one(c, p, g, m, v):
    b1, b2, t = ADAMW["beta1"], c["beta2"], c["step"]
    m1 = m + (1.0 - b1) * (g - m)
    v1 = v + (1.0 - b2) * (g * g - v)
    mhat, vhat = m1 / (1.0 - b1 ** t), v1 / (1.0 - b2 ** t)
    return p - ADAMW["lr"] * (mhat / (torch.sqrt(vhat) + ADAMW["eps"]) + ADAMW["weight_decay"] * p), m1, v1


def _exact_adamw(st):
    c = st["case"]
    parts = []
    span = 2 ** 26   # a multiple of the block
    for a in range(0, st["p"].numel(), span):
        p, g, m, v = (st[name][a:a + span] for name in ("p", "g", "m", "v"))
        if c["state"] == "e4m3":
            at = torch.arange(m.numel(), device="cuda") // BLOCK + a // BLOCK
            m = m.float().double() * st["ms"].double()[at]
            v = (v.float().double() * st["vs"].double()[at]) ** 2
        p1, m1, v1 = _exact_adamw_one(c, p.double(), g.double(), m.double(), v.double())
        if c["state"] == "e4m3":
            (mq, ms), (vq, vs) = _exact_blocks(m1, False), _exact_blocks(torch.sqrt(v1), True)
            parts.append((p1, mq.float(), vq.float(), ms, vs))
        else:
            parts.append((p1, m1, v1))
    out = {name: torch.cat(got) for name, got in zip(("p", "m", "v", "ms", "vs"), zip(*parts))}
    if c["copy"]:
        out["copy"] = out["p"]
    return out


def _exact_policy(st):
    c = st["case"]
    val = {k: st[k].double().cpu().numpy() for k in ("logp", "old", "adv")}
    ref = st["ref"].double().cpu().numpy() if c["ref"] else None
    ok, cu = st["targets"].cpu().numpy() >= 0, st["cu"].cpu().numpy()
    sequences = cu.size - 1
    loss, grad, stats = 0.0, np.zeros(c["n"]), np.zeros(4)
    total = sum(int(ok[a:b].sum()) for a, b in zip(cu[:-1], cu[1:]))
    for s in range(sequences):
        at = cu[s] + np.flatnonzero(ok[cu[s]:cu[s + 1]])
        if at.size == 0:
            continue
        x = val["logp"][at]
        a = val["adv"][at] if c["advantage"] == "token" else np.full(at.size, val["adv"][s])
        r = np.exp(x - val["old"][at])
        free = r * a
        held = np.clip(r, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * a
        gain = np.minimum(free, held)
        stop = free > held
        if c["dual_clip"]:
            low = (a < 0) & (r > c["dual_clip"])
            gain = np.where(low, c["dual_clip"] * a, gain)
            stop |= low
        each, slope, kl = -gain, np.where(stop, 0.0, -free), np.zeros(at.size)
        if ref is not None:
            d = x - ref[at]
            kl = {"k1": d, "k2": 0.5 * d * d, "k3": np.exp(-d) - 1.0 + d}[c["kl"]]
            each = each + KL_WEIGHT * kl
            slope = slope + KL_WEIGHT * {"k1": np.ones_like(d), "k2": d, "k3": 1.0 - np.exp(-d)}[c["kl"]]
        w = {"mean": 1.0 / total, "sum": 1.0, "sequence_mean": 1.0 / (sequences * at.size)}[c["reduction"]]
        loss += w * float(each.sum())
        grad[at] = w * slope
        # a token without advantage counts as clipped above, where its slope is nil anyway
        stop |= (a == 0) & (r > 1.0 + CLIP_HIGH)
        stats += [kl.sum(), stop.sum(), r.sum(), (1.0 / r - 1.0 + np.log(r)).sum()]
    return torch.tensor(loss, dtype=torch.float64), torch.from_numpy(stats / max(total, 1)), torch.from_numpy(grad)


def _exact_preference(st):
    c = st["case"]
    x = st["logp"].double().cpu().numpy()
    if c["ref"]:
        x = x - st["ref"].double().cpu().numpy()
    ok, cu, beta, pairs = st["targets"].cpu().numpy() >= 0, st["cu"].cpu().numpy(), BETA[c["kind"]], c["pairs"]
    at = [cu[q] + np.flatnonzero(ok[cu[q]:cu[q + 1]]) for q in range(2 * pairs)]
    part = [1.0 / max(1, a.size) if c["average"] else 1.0 for a in at]
    s = np.array([x[a].sum() * f for a, f in zip(at, part)])
    loss, grad = 0.0, np.zeros(c["n"])
    for j in range(pairs):
        h = beta * (s[j] - s[pairs + j])
        if c["kind"] == "sigmoid":
            loss += (1.0 - SMOOTH) * np.logaddexp(0.0, -h) + SMOOTH * np.logaddexp(0.0, h)
            slope = SMOOTH / (1.0 + math.exp(-h)) - (1.0 - SMOOTH) / (1.0 + math.exp(h))
        elif c["kind"] == "hinge":
            loss += max(0.0, 1.0 - h)
            slope = -1.0 if h < 1.0 else 0.0
        else:
            loss += ((h - 0.5) / beta) ** 2
            slope = 2.0 * (h - 0.5) / beta ** 2
        grad[at[j]] = beta * slope * part[j] / pairs
        grad[at[pairs + j]] = -beta * slope * part[pairs + j] / pairs
    return torch.tensor(loss / pairs, dtype=torch.float64), torch.from_numpy(beta * s), torch.from_numpy(grad)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        ids = st["ids"].long()
        keep = torch.nonzero(ids >= 0)[:, 0]
        out = torch.zeros(case["n"], case["hidden"], dtype=torch.float64, device="cuda")
        rows = st["w"][ids[keep]].float().double() * case["scale"]
        if case["weight"] == "e4m3":
            rows *= st["ws"].double()[ids[keep] // BLOCK].repeat_interleave(BLOCK, 1)
        out[keep] = rows
        return out
    if op == "embed_grad":
        ids = st["ids"].long()
        keep = torch.nonzero(ids >= 0)[:, 0]
        each, back = torch.unique(ids[keep], return_inverse=True)
        sums = torch.zeros(each.numel(), case["hidden"], dtype=torch.float64, device="cuda")
        sums.index_add_(0, back, st["dy"][keep].double() * case["scale"])
        if "acc" in st:
            out = st["acc"].double()
        else:
            out = torch.zeros(case["vocab"], case["hidden"], dtype=torch.float64, device="cuda")
        out[each] += sums
        return out
    return {"policy": _exact_policy, "preference": _exact_preference, "adamw": _exact_adamw}[op](st)
