"""Plain 64-bit definitions of the operators in include/lmhead_train.h, on the
CPU, written from the formulas and sharing no code with the library."""
import math

import numpy as np

E4M3_MAX = 448.0


def embedding(ids, w, scale):
    out = np.zeros((len(ids), w.shape[1]))
    for i, v in enumerate(ids):
        if v >= w.shape[0]:
            out[i] = np.nan
        elif v >= 0:
            out[i] = w[v] * scale
    return out


def embedding_grad(ids, dout, vocab, scale):
    """(sums, sums of magnitudes, tokens of each id)."""
    s, a, c = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1])), np.zeros(vocab)
    keep = (ids >= 0) & (ids < vocab)
    np.add.at(s, ids[keep], dout[keep] * scale)
    np.add.at(a, ids[keep], np.abs(dout[keep] * scale))
    np.add.at(c, ids[keep], 1)
    return s, a, c


def counted(n, targets, cu):
    """(sequence of each token or -1, whether it counts)."""
    seq = np.full(n, -1)
    for s in range(len(cu) - 1):
        seq[cu[s]:cu[s + 1]] = s
    ok = seq >= 0
    if targets is not None:
        ok &= targets >= 0
    return seq, ok


def policy(logp, adv, old=None, ref=None, targets=None, cu=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0,
           kl_weight=0.0, kl_kind="k3", reduction="mean", num_valid=-1, per_sequence=False):
    """(loss, stats, dlogp for an upstream gradient of 1, per-token size of the
    terms that dlogp is made of)."""
    n = len(logp)
    cu = np.array([0, n]) if cu is None else cu
    sequences = len(cu) - 1
    seq, ok = counted(n, targets, cu)
    loss, dlogp, size, stats = 0.0, np.zeros(n), np.zeros(n), np.zeros(4)
    total = int(ok.sum())
    for s in range(sequences):
        at = np.flatnonzero(ok & (seq == s))
        if reduction == "mean":
            den = total if num_valid < 0 else num_valid
        elif reduction == "sum":
            den = 1
        else:
            den = (sequences if num_valid < 0 else num_valid) * len(at)
        w = 1.0 / den if den else 0.0
        for t in at:
            a = adv[s] if per_sequence else adv[t]
            d = logp[t] - old[t] if old is not None else 0.0
            r = math.exp(d)
            if a >= 0:
                clipped = r > 1 + clip_high
                rho = min(r, 1 + clip_high)
            else:
                clipped = r < 1 - clip_low
                rho = max(r, 1 - clip_low)
                if dual_clip and rho > dual_clip:
                    clipped, rho = True, dual_clip
            k = dk = 0.0
            if ref is not None:
                x = logp[t] - ref[t]
                k, dk = {"k1": (x, 1.0), "k2": (x * x / 2, x), "k3": (math.expm1(-x) + x, -math.expm1(-x))}[kl_kind]
            loss += w * (-a * rho + kl_weight * k) if w else 0.0
            dlogp[t] = w * ((0.0 if clipped else -a * r) + kl_weight * dk)
            grow = abs(x) * math.exp(-x) if ref is not None else 0.0
            size[t] = w * (abs(a) * r * (4 + abs(d)) + abs(kl_weight) * (4 * abs(dk) + grow))
            stats += [k, clipped, r, math.expm1(-d) + d]
    return loss, stats / max(total, 1), dlogp, size


def preference(logp, cu, ref=None, targets=None, kind="sigmoid", beta=0.1, margin=0.0, label_smoothing=0.0,
               average=False, num_pairs=-1):
    """(loss, rewards, dlogp)."""
    n, pairs = len(logp), (len(cu) - 1) // 2
    seq, ok = counted(n, targets, cu)
    gain = logp - ref if ref is not None else logp
    at = [np.flatnonzero(ok & (seq == s)) for s in range(2 * pairs)]
    f = np.array([1.0 / len(a) if average and len(a) else 1.0 for a in at])
    s = np.array([math.fsum(gain[a]) for a in at]) * f
    den = pairs if num_pairs < 0 else num_pairs
    loss, dlogp = 0.0, np.zeros(n)
    for j in range(pairs):
        h = beta * (s[j] - s[pairs + j]) - margin
        if kind == "sigmoid":
            each = (1 - label_smoothing) * np.logaddexp(0, -h) + label_smoothing * np.logaddexp(0, h)
            slope = -(1 - label_smoothing) * math.exp(-np.logaddexp(0, h)) + \
                label_smoothing * math.exp(-np.logaddexp(0, -h))
        elif kind == "hinge":
            each, slope = max(0.0, 1 - h), -1.0 if h < 1 else 0.0
        else:
            each, slope = ((h - 0.5) / beta) ** 2, 2 * (h - 0.5) / beta ** 2
        if den:
            loss += each / den
            dlogp[at[j]] = beta * slope * f[j] / den
            dlogp[at[pairs + j]] = -beta * slope * f[pairs + j] / den
    return loss, beta * s, dlogp


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay):
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v / (1 - beta2 ** step)) + eps
    return p - lr * weight_decay * p - lr * m / (1 - beta1 ** step) / den, m, v, den


def block_scale(x):
    """Scale of each value's block of 128 consecutive ones."""
    full = np.zeros(-(-len(x) // 128) * 128)
    full[:len(x)] = np.abs(x)
    amax = full.reshape(-1, 128).max(1)
    s = np.where(amax > 0, np.maximum(amax / E4M3_MAX, 2.0 ** -126), 1.0)
    return s, np.repeat(s, 128)[:len(x)]
