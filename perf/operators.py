"""Measured cases of the answer path: final RMS norm (with the residual's
addition, bf16 or 8-bit output, and its backward), logits in 8-bit floating
point with block scales, the block quantiser, and next-token sampling.

``own`` chooses between the plain torch form (fp32, or fp64 where a border
decides) and the library's kernels; both take what ``prepare`` gives.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # one decoded token: the final norm of a single row (latency)
        dict(name="norm_quant_1", op="norm_quant", n=1, hidden=4096, eps=1e-6, offset=0.0, residual=True),
        # a prefill's or a large batch's rows
        dict(name="norm_quant_8192", op="norm_quant", n=8192, hidden=4096, eps=1e-6, offset=0.0, residual=True),
        # the training step's norm in front of the log-prob entry: forward and backward
        dict(name="norm_train_16384", op="norm_train", n=16384, hidden=4096, eps=1e-6, offset=0.0, residual=True,
             weight="bf16"),
        # the same with few rows, an odd count, a zero-centred fp32 weight and no residual
        dict(name="norm_train_777", op="norm_train", n=777, hidden=2048, eps=1e-5, offset=1.0, residual=False,
             weight="fp32"),
        # a head's rows quantised as they come (no norm of their own)
        dict(name="quant_rows_300", op="quant", rows=300, cols=2048, block_rows=1),
        # a vocabulary matrix quantised once, as after loading or an optimiser step
        dict(name="quant_weight_151936", op="quant", rows=151936, cols=4096, block_rows=128),
        # one decoded token's logits
        dict(name="logits_1", op="logits", n=1, vocab=151936, hidden=4096, out="fp32"),
        # a decode batch
        dict(name="logits_64", op="logits", n=64, vocab=128256, hidden=4096, out="fp32"),
        # rows to score or verify: the matrix product decides
        dict(name="logits_2048", op="logits", n=2048, vocab=151936, hidden=4096, out="bf16"),
        # one chat stream: temperature, top-k and top-p together
        dict(name="sample_1", op="sample", n=1, vocab=151936, logits="fp32", spread=2.5, mode="chat"),
        # a decode batch whose requests differ; masked tokens, one row with nothing left
        dict(name="sample_64", op="sample", n=64, vocab=128256, logits="bf16", spread=2.0, mode="mixed"),
        # rollouts: nucleus sampling over wide distributions
        dict(name="sample_256", op="sample", n=256, vocab=151936, logits="fp32", spread=1.3, mode="nucleus"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_quant", "norm_train", "quant", "logits", "logits", "sample", "sample"])
    if op in ("norm_quant", "norm_train"):
        hidden = 128 * _log_int(rng, 2, 64)
        n = _log_int(rng, 1, 8192 * 4096 // hidden)
        c = dict(op=op, n=n, hidden=hidden, eps=rng.choice([1e-6, 1e-5]), offset=rng.choice([0.0, 1.0]),
                 residual=rng.random() < 0.7)
        if op == "norm_train":
            c["weight"] = rng.choice(["bf16", "fp32"])
        return c
    if op == "quant":
        cols = 128 * _log_int(rng, 2, 64)
        return dict(op=op, rows=_log_int(rng, 1, 2 ** 28 // cols), cols=cols, block_rows=rng.choice([1, 128]))
    if op == "logits":
        hidden = 128 * _log_int(rng, 2, 40)
        vocab = _log_int(rng, 1000, 151936)
        n = _log_int(rng, 1, 2048)
        return dict(op=op, n=n, vocab=vocab, hidden=hidden, out=rng.choice(["fp32", "bf16"]))
    vocab = _log_int(rng, 1000, 151936)
    return dict(op=op, n=_log_int(rng, 1, 256), vocab=vocab, logits=rng.choice(["fp32", "bf16"]),
                spread=round(rng.uniform(1.0, 4.0), 3), mode=rng.choice(["chat", "mixed", "nucleus", "plain", "min_p"]))


# ------------------------------------------------------------------ inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _blocks_quantised(rows, cols, block_rows, std, g):
    """Quantised values and scales as a user's loaded weights or rows have them."""
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(-(-rows // block_rows), cols // BLOCK, dtype=torch.float32, device="cuda")
    step = 128 * 128
    for r0 in range(0, rows, step):
        r1 = min(rows, r0 + step)
        x = _normal((r1 - r0, cols), g, std)
        amax = x.abs().view(r1 - r0, cols // BLOCK, BLOCK).amax(2)
        if block_rows > 1:
            pad = -(r1 - r0) % block_rows
            amax = torch.nn.functional.pad(amax, (0, 0, 0, pad)).view(-1, block_rows, cols // BLOCK).amax(1)
        scale = amax / E4M3_MAX
        s[r0 // block_rows:r0 // block_rows + scale.shape[0]] = scale
        each = scale.repeat_interleave(block_rows, 0)[:r1 - r0].repeat_interleave(BLOCK, 1)
        q[r0:r1] = (x / each).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm_quant", "norm_train"):
        n, h = case["n"], case["hidden"]
        bf = torch.bfloat16
        wt = torch.float32 if case.get("weight") == "fp32" else bf
        st = dict(case=case, x=_normal((n, h), g).to(bf),
                  res=_normal((n, h), g, 3.0).to(bf) if case["residual"] else None,
                  w=(1.0 - case["offset"] + _normal((h,), g, 0.1)).to(wt))
        if op == "norm_train":
            st["dy"] = _normal((n, h), g, 0.01).to(bf)
            st["dr"] = _normal((n, h), g, 0.01).to(bf) if case["residual"] else None
        return st
    if op == "quant":
        return dict(case=case, x=_normal((case["rows"], case["cols"]), g, 0.02).to(torch.bfloat16))
    if op == "logits":
        a, sa = _blocks_quantised(case["n"], case["hidden"], 1, 1.0, g)
        w, sw = _blocks_quantised(case["vocab"], case["hidden"], 128, 0.02, g)
        return dict(case=case, a=a, sa=sa, w=w, sw=sw)
    n, v, mode = case["n"], case["vocab"], case["mode"]
    x = _normal((n, v), g, case["spread"])
    # a few tokens stand out, as after a real context
    top = torch.randint(0, v, (n, 24), generator=g, device="cuda")
    x.scatter_add_(1, top, _normal((n, 24), g).abs() * 2.0 * case["spread"])
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float32).clamp(max=1.0 - 2.0 ** -24)
    row = torch.rand(4, n, generator=g, device="cuda", dtype=torch.float32)
    st = dict(case=case, u=u, temperature=None, top_k=None, top_p=None, min_p=None)
    if mode == "chat":
        st.update(temperature=torch.full((n,), 0.7, device="cuda"),
                  top_k=torch.full((n,), 50, dtype=torch.int32, device="cuda"),
                  top_p=torch.full((n,), 0.9, device="cuda"))
    elif mode == "nucleus":
        st.update(top_p=torch.full((n,), 0.95, device="cuda"))
    elif mode == "min_p":
        st.update(temperature=0.5 + row[0], min_p=0.02 + 0.1 * row[1])
    elif mode == "mixed":
        off = row[3]
        st.update(temperature=0.3 + 1.2 * row[0],
                  top_k=torch.where(off < 0.3, 0.0, 1.0 + 200.0 * row[1]).to(torch.int32),
                  top_p=torch.where((off > 0.2) & (off < 0.5), 1.0, 0.5 + 0.5 * row[2]),
                  min_p=torch.where(off > 0.7, 0.1 * row[1], 0.0))
        # a grammar leaves a tenth of the tokens in every fourth row, and none in one
        gone = torch.rand(v, generator=g, device="cuda") < 0.9
        x[::4] = x[::4].masked_fill(gone, float("-inf"))
        x[n // 2] = float("-inf")
    st["logits"] = x if case["logits"] == "fp32" else x.to(torch.bfloat16)
    return st


# -------------------------------------------------------------- plain forms

def _plain_norm(st):
    c = st["case"]
    x = st["x"].float()
    if st["res"] is not None:
        r = (x + st["res"].float()).to(torch.bfloat16)
    else:
        r = st["x"]
    rf = r.float()
    rstd = torch.rsqrt(rf.square().mean(1) + c["eps"])
    y = rf * rstd[:, None] * (c["offset"] + st["w"].float())
    return r, rstd, y


def _plain_quant(y, block_rows):
    rows, cols = y.shape
    amax = y.abs().view(rows, cols // BLOCK, BLOCK).amax(2)
    if block_rows > 1:
        amax = torch.nn.functional.pad(amax, (0, 0, 0, -rows % block_rows))
        amax = amax.view(-1, block_rows, cols // BLOCK).amax(1)
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    each = scale.repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else scale
    q = (y.view(rows, cols // BLOCK, BLOCK) / each[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(rows, cols).to(torch.float8_e4m3fn), scale


def _plain_norm_train(st):
    c = st["case"]
    r, rstd, y = _plain_norm(st)
    dy = st["dy"].float()
    xh = r.float() * rstd[:, None]
    g = dy * (c["offset"] + st["w"].float())
    dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if st["dr"] is not None:
        dx = dx + st["dr"].float()
    dw = (dy * xh).sum(0)
    out = (y.to(torch.bfloat16), dx.to(torch.bfloat16), dw.to(st["w"].dtype))
    return out + (r,) if st["res"] is not None else out


def _plain_logits(st):
    a, w = st["a"], st["w"]
    af = (a.float().view(a.shape[0], -1, BLOCK) * st["sa"][:, :, None]).view(a.shape)
    sw = st["sw"].repeat_interleave(BLOCK, 0)[:w.shape[0]]
    wf = (w.float().view(w.shape[0], -1, BLOCK) * sw[:, :, None]).view(w.shape)
    z = af @ wf.t()
    return z if st["case"]["out"] == "fp32" else z.to(torch.bfloat16)


def _plain_sample(st):
    x = st["logits"].double()
    n, v = x.shape
    valid = x > -math.inf
    top = x.amax(1, keepdim=True)
    d = x - torch.where(top > -math.inf, top, 0.0)
    if st["temperature"] is not None:
        d = d / st["temperature"].double()[:, None]
    w = torch.where(valid, d.exp(), 0.0)
    keep = valid
    if st["top_k"] is not None or st["top_p"] is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        ws, ks = w.gather(1, order), valid.gather(1, order)
        rank = torch.arange(v, device=x.device)[None]
        if st["top_k"] is not None:
            k = st["top_k"].long()[:, None]
            ks = ks & ((k <= 0) | (rank < k))
        if st["top_p"] is not None:
            wk = torch.where(ks, ws, 0.0)
            before = wk.cumsum(1) - wk
            p = st["top_p"].double()[:, None]
            ks = ks & ((p >= 1.0) | (rank == 0) | (before < p * wk.sum(1, keepdim=True)))
        keep = torch.zeros_like(valid).scatter_(1, order, ks)
    if st["min_p"] is not None:
        keep = keep & (w >= st["min_p"].double()[:, None])
    run_w = torch.where(keep, w, 0.0).cumsum(1)
    total = run_w[:, -1:]
    token = (run_w <= st["u"].double()[:, None] * total).sum(1)
    last = (run_w < total).sum(1)
    token = torch.minimum(token, last).clamp(max=v - 1)
    lp = d.gather(1, token[:, None])[:, 0] - w.sum(1).log()
    empty = ~valid.any(1)
    return (torch.where(empty, -1, token).to(torch.int32), torch.where(empty, 0.0, lp).float())


# ------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import chunked_lm_head_amd as lm
        if op == "norm_quant":
            q, scale, r = lm.rms_norm_quant(state["x"], state["w"], state["res"], eps=c["eps"],
                                            weight_offset=c["offset"])
            return (q, scale, r) if state["res"] is not None else (q, scale)
        if op == "norm_train":
            f = lm.rms_norm_forward(state["x"], state["w"], state["res"], eps=c["eps"], weight_offset=c["offset"])
            r = f.residual_out if state["res"] is not None else state["x"]
            dx, dw = lm.rms_norm_backward(state["dy"], r, state["w"], f.rstd, dresidual=state["dr"],
                                          weight_offset=c["offset"])
            return (f.y, dx, dw, r) if state["res"] is not None else (f.y, dx, dw)
        if op == "quant":
            return lm.quantize_fp8(state["x"], block_rows=c["block_rows"])
        if op == "logits":
            return lm.logits_fp8(state["a"], state["sa"], state["w"], state["sw"],
                                 out_dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16)
        return lm.sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                         top_p=state["top_p"], min_p=state["min_p"])
    if op == "norm_quant":
        r, _, y = _plain_norm(state)
        q, scale = _plain_quant(y, 1)
        return (q, scale, r) if state["res"] is not None else (q, scale)
    if op == "norm_train":
        return _plain_norm_train(state)
    if op == "quant":
        return _plain_quant(state["x"].float(), c["block_rows"])
    if op == "logits":
        return _plain_logits(state)
    return _plain_sample(state)


def work(case):
    op = case["op"]
    if op in ("norm_quant", "norm_train"):
        n, h, res = case["n"], case["hidden"], 1 if case["residual"] else 0
        if op == "norm_quant":
            return dict(bytes=n * h * (2 + 4 * res + 1) + 4 * n * h // BLOCK + 2 * h, flops=7 * n * h)
        # x, dy in and y, dx out; with a residual also res, dr in and the new residual out
        wb = 4 if case["weight"] == "fp32" else 2
        return dict(bytes=2 * n * h * (4 + 3 * res) + 2 * wb * h, flops=16 * n * h)
    if op == "quant":
        r, k = case["rows"], case["cols"]
        return dict(bytes=3 * r * k + 4 * -(-r // case["block_rows"]) * k // BLOCK, flops=3 * r * k)
    if op == "logits":
        n, v, h = case["n"], case["vocab"], case["hidden"]
        return dict(bytes=n * h + v * h + 4 * (n + -(-v // BLOCK)) * h // BLOCK + n * v * (4 if case["out"] == "fp32" else 2),
                    flops=2 * n * v * h)
    n, v = case["n"], case["vocab"]
    return dict(bytes=n * v * (4 if case["logits"] == "fp32" else 2), flops=4 * n * v)


# ------------------------------------------------------ definition, 64 bits

def _e4m3_64(y):
    """Nearest e4m3 value (ties to even) of fp64 values within +-448."""
    mag = y.abs()
    e = torch.floor(torch.log2(torch.where(mag > 0, mag, 1.0))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(y) * torch.clamp(torch.round(mag / step) * step, max=E4M3_MAX)


def _exact_scaled(y, block_rows):
    rows, cols = y.shape
    nb = -(-rows // block_rows)
    scale = torch.empty(nb, cols // BLOCK, dtype=torch.float64, device=y.device)
    q = torch.empty_like(y)
    span = max(1, 4096 // block_rows)
    for b0 in range(0, nb, span):
        b1 = min(nb, b0 + span)
        part = y[b0 * block_rows:min(rows, b1 * block_rows)]
        full = torch.zeros((b1 - b0) * block_rows, cols, dtype=y.dtype, device=y.device)
        full[:part.shape[0]] = part
        blk = full.view(b1 - b0, block_rows, cols // BLOCK, BLOCK)
        s = blk.abs().amax((1, 3)) / E4M3_MAX
        s[s == 0] = 1.0
        scale[b0:b1] = s
        got = _e4m3_64(blk / s[:, None, :, None]).view(-1, cols)
        q[b0 * block_rows:b0 * block_rows + part.shape[0]] = got[:part.shape[0]]
    return q, scale


def _exact_norm(st):
    c = st["case"]
    r64 = st["x"].double()
    if st["res"] is not None:
        r64 = r64 + st["res"].double()
        r64 = r64.to(torch.bfloat16).double()   # the residual stream is held in bf16: part of the definition
    inv = 1.0 / torch.sqrt((r64 * r64).sum(1, keepdim=True) / r64.shape[1] + c["eps"])
    return r64, inv, st["w"].double() + c["offset"]


def _exact_sample_row(x, u, tau, k, p, min_p):
    ids = np.flatnonzero(x > -np.inf)
    if ids.size == 0:
        return -1, 0.0
    z = (x[ids] - x[ids].max()) / tau
    w = np.exp(z)
    lse = math.log(math.fsum(w.tolist()))
    kept = np.argsort(-x[ids], kind="stable")
    if k > 0:
        kept = kept[:k]
    if p < 1.0:
        run = np.cumsum(w[kept])
        kept = kept[:int(np.searchsorted(run, p * run[-1], side="left")) + 1]
    kept = np.sort(kept[w[kept] >= min_p])
    run = np.cumsum(w[kept])
    j = min(int(np.searchsorted(run, u * run[-1], side="right")), kept.size - 1)
    return int(ids[kept[j]]), float(z[kept[j]] - lse)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_quant":
        r, inv, w = _exact_norm(st)
        q, scale = _exact_scaled(r * inv * w, 1)
        return (q, scale, r) if st["res"] is not None else (q, scale)
    if op == "norm_train":
        r, inv, w = _exact_norm(st)
        dy = st["dy"].double()
        # dL/dr of y_j = r_j inv w_j, inv = (sum r^2 / h + eps)^-1/2
        dot = (dy * w * r).sum(1, keepdim=True)
        dx = inv * w * dy - r * inv ** 3 * dot / r.shape[1]
        if st["dr"] is not None:
            dx = dx + st["dr"].double()
        out = (r * inv * w, dx, (dy * r * inv).sum(0))
        return out + (r,) if st["res"] is not None else out
    if op == "quant":
        if case["rows"] * case["cols"] > 2 ** 27:
            # amax and the rounding by pieces of rows, the same definition
            qs = [_exact_scaled(st["x"][r0:r0 + 16384].double(), case["block_rows"])
                  for r0 in range(0, case["rows"], 16384)]
            return torch.cat([q.float() for q, _ in qs]), torch.cat([s for _, s in qs])
        return _exact_scaled(st["x"].double(), case["block_rows"])
    if op == "logits":
        n, v, h = case["n"], case["vocab"], case["hidden"]
        a = st["a"].double() * st["sa"].double().repeat_interleave(BLOCK, 1)
        z = torch.empty(n, v, dtype=torch.float64, device="cuda")
        for v0 in range(0, v, 128 * 128):
            v1 = min(v, v0 + 128 * 128)
            sw = st["sw"][v0 // BLOCK:-(-v1 // BLOCK)].double()
            sw = sw.repeat_interleave(BLOCK, 0)[:v1 - v0].repeat_interleave(BLOCK, 1)
            z[:, v0:v1] = a @ (st["w"][v0:v1].double() * sw).t()
        return z
    x = st["logits"].double().cpu().numpy()
    n = case["n"]
    col = lambda name, off: st[name].double().cpu().numpy() if st[name] is not None else np.full(n, off)  # noqa: E731
    u, tau, k, p, mp = st["u"].double().cpu().numpy(), col("temperature", 1.0), col("top_k", 0), col("top_p", 1.0), \
        col("min_p", 0.0)
    got = [_exact_sample_row(x[i], u[i], tau[i], int(k[i]), p[i], mp[i]) for i in range(n)]
    return (torch.tensor([t for t, _ in got], dtype=torch.int32), torch.tensor([lp for _, lp in got], dtype=torch.float64))
