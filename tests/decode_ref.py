"""Plain 64-bit definitions of the operators in include/lmhead_decode.h, on the
CPU, written from the formulas and sharing no code with the library."""
import math

import numpy as np

E4M3_MAX = 448.0


def bf16_round(x):
    """fp64/fp32 -> nearest bf16 (ties to even) of the fp32 value, as fp64."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def norm(x, res, w, eps, offset):
    """(r, rstd, y) in fp64; r is the bf16 residual stream."""
    r = x if res is None else bf16_round(x.astype(np.float32) + res.astype(np.float32))
    rstd = 1.0 / np.sqrt((r * r).mean(1) + eps)
    return r, rstd, r * rstd[:, None] * (offset + w)


def norm_backward(dy, r, w, rstd, dres, offset):
    g = dy * (offset + w)
    h = r * rstd[:, None]
    dx = rstd[:, None] * (g - h * (g * h).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    return dx, (dy * h).sum(0)


def block_scales(x, block_rows):
    rows, cols = x.shape
    nb = -(-rows // block_rows)
    full = np.zeros((nb * block_rows, cols))
    full[:rows] = np.abs(x)
    amax = full.reshape(nb, block_rows, cols // 128, 128).max((1, 3))
    return np.where(amax > 0, np.maximum(amax / E4M3_MAX, 2.0 ** -126), 1.0)


def spread_scales(s, block_rows, rows):
    return np.repeat(np.repeat(s, block_rows, 0)[:rows], 128, 1)


def sample_row(x, u, tau=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row of fp64 logits by the documented rule."""
    ids = np.flatnonzero(x > -np.inf)
    if ids.size == 0:
        return -1, 0.0
    z = (x[ids] - x[ids].max()) / tau
    w = np.exp(z)
    lse = math.log(math.fsum(w.tolist()))
    order = np.argsort(-x[ids], kind="stable")
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1.0:
        run = np.cumsum(w[order])
        keep = (run - w[order]) < top_p * run[-1]
        keep[0] = True
        order = order[keep]
    kept = np.sort(order[w[order] >= min_p])
    run = np.cumsum(w[kept])
    j = min(int((run <= u * run[-1]).sum()), kept.size - 1)
    return int(ids[kept[j]]), float(z[kept[j]] - lse)


def sample(x, u, tau=None, top_k=None, top_p=None, min_p=None):
    n = x.shape[0]

    def per_row(v, off):
        return np.full(n, off) if v is None else np.broadcast_to(np.asarray(v, dtype=np.float64), (n,))
    tau, k, p, m = per_row(tau, 1.0), per_row(top_k, 0), per_row(top_p, 1.0), per_row(min_p, 0.0)
    got = [sample_row(x[i], float(u[i]), float(tau[i]), int(k[i]), float(p[i]), float(m[i])) for i in range(n)]
    return np.array([t for t, _ in got], dtype=np.int64), np.array([v for _, v in got])
