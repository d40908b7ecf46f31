"""The policy loss and the preference loss on packed tokens against the plain
64-bit definitions."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def dev(x, dtype=torch.float32):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def f32(x):
    return x.astype(np.float32).astype(np.float64)


def lengths(rng, n, sequences, kind):
    if kind == "even":
        cu = np.linspace(0, n, sequences + 1).astype(int)
    elif kind == "empty":   # empty ones in front, within and behind; tokens outside
        cu = np.sort(np.concatenate([[0, 0], rng.integers(0, n + 1, sequences - 1)])) if sequences > 1 else np.array([0, n])
        cu = np.minimum(cu, max(0, n - n // 8))
    else:                   # one long one, the others of a few tokens
        cu = np.concatenate([np.minimum(np.arange(sequences), n), [n]])
    return cu


def inputs(n, sequences, kind, seed, off=0.3):
    rng = np.random.default_rng(seed)
    cu = lengths(rng, n, sequences, kind)
    targets = np.where(rng.random(n) < off, -rng.integers(1, 200, n), rng.integers(0, 1000, n))
    if sequences > 2:   # a sequence whose tokens are all ignored
        s = sequences // 2
        targets[cu[s]:cu[s + 1]] = -100
    logp = f32(-np.abs(rng.standard_normal(n)) * 1.5)
    old, ref_ = f32(logp + 0.2 * rng.standard_normal(n)), f32(logp + 0.4 * rng.standard_normal(n))
    return rng, cu, targets, logp, old, ref_


SIZES = [(1, 1), (2, 2), (63, 4), (1000, 7), (8192, 3), (8193, 5), (9000, 2500), (50001, 300)]


@pytest.mark.parametrize("n,sequences", SIZES)
@pytest.mark.parametrize("kind", ["even", "empty", "skewed"])
@pytest.mark.parametrize("reduction", ["mean", "sum", "sequence_mean"])
def test_policy(n, sequences, kind, reduction):
    rng, cu, targets, logp, old, ref_ = inputs(n, sequences, kind, n + sequences)
    per = bool(n % 2)
    adv = f32(rng.standard_normal(sequences if per else n))
    kw = dict(clip_low=0.15, clip_high=0.25, dual_clip=1.3 if n % 3 == 0 else 0.0, kl_weight=0.3,
              kl_kind=["k1", "k2", "k3"][(n + sequences) % 3], reduction=reduction)
    want = ref.policy(logp, adv, old, ref_, targets, cu, per_sequence=per, **kw)
    args = (dev(logp), dev(adv), dev(old), dev(ref_), dev(targets, torch.int32), dev(cu, torch.int32))
    f = lm.policy_loss_forward(*args, advantage_per_sequence=per, **kw)
    check_policy(f, want, logp, adv, old, ref_, targets, cu, per, kw)
    grad = torch.tensor([-1.5], device="cuda")
    got = lm.policy_loss_backward(grad, f.weights, *args, advantage_per_sequence=per, **kw)
    g = -1.5 * want[2]
    # the terms' roundings (size counts them), the weight, two products and sums
    assert (np.abs(got.double().cpu().numpy() - g) <= 1.5 * U * (want[3] + 4 * np.abs(want[2])) * 1.01).all()
    assert (got.cpu().numpy()[~ref.counted(n, targets, cu)[1]] == 0).all()
    again = lm.policy_loss_forward(*args, advantage_per_sequence=per, **kw)
    assert all(torch.equal(a, b) for a, b in zip(f, again))


def check_policy(f, want, logp, adv, old, ref_, targets, cu, per, kw):
    n = len(logp)
    seq, ok = ref.counted(n, targets, cu)
    total = max(1, int(ok.sum()))
    a = np.abs(adv[np.clip(seq, 0, len(cu) - 2)] if per else adv)
    d, x = logp - old, logp - ref_
    r = np.exp(d)
    # of a token: the ratio's roundings, the products and the KL estimate's (a
    # difference of terms up to 1 + e^-x outside the series)
    err = U * (a * r * (4 + np.abs(d)) + kw["kl_weight"] * (4 + 4 * np.abs(x) + 4 * np.exp(-x)))
    w = np.zeros(n)
    counts = np.array([(ok & (seq == s)).sum() for s in range(len(cu) - 1)])
    for s in range(len(cu) - 1):
        den = {"mean": total, "sum": 1, "sequence_mean": (len(cu) - 1) * max(1, counts[s])}[kw["reduction"]]
        w[seq == s] = 1.0 / den
    tol = (w * err)[ok].sum() * 1.01 + U * abs(want[0]) + 1e-300
    assert abs(float(f.loss) - want[0]) <= tol
    stats = f.stats.double().cpu().numpy()
    assert abs(stats[0] - want[1][0]) <= U * ((4 + 4 * np.abs(x) + 4 * np.exp(-x))[ok].sum() / total + abs(want[1][0]))
    assert abs(stats[1] - want[1][1]) <= U * want[1][1] * 1.01   # a count over a count
    assert abs(stats[2] - want[1][2]) <= U * ((r * (4 + np.abs(d)))[ok].sum() / total + want[1][2])
    assert abs(stats[3] - want[1][3]) <= U * ((4 + 4 * np.abs(d) + 4 * np.exp(-d))[ok].sum() / total + want[1][3])
    got = f.weights.double().cpu().numpy()
    if kw["reduction"] == "sequence_mean":
        full = np.where(counts > 0, 1.0 / ((len(cu) - 1) * np.maximum(counts, 1)), 0.0)
    else:
        full = np.full(len(cu) - 1, (1.0 / total if ok.any() else 0.0) if kw["reduction"] == "mean" else 1.0)
    assert (np.abs(got - full) <= U * full * 1.01).all()


@pytest.mark.parametrize("n", [0, 5, 20000])
def test_policy_plain_forms(n):
    """No sequences, no targets, no old log-probs, no reference; given counts."""
    rng = np.random.default_rng(n)
    logp, adv = f32(-rng.random(n)), f32(rng.standard_normal(n))
    x, a = dev(logp), dev(adv)
    one = torch.ones((), device="cuda")
    f = lm.policy_loss_forward(x, a)
    size = np.abs(adv).sum() / max(n, 1)
    assert abs(float(f.loss) - (-adv.mean() if n else 0.0)) <= 4 * U * size
    assert f.stats.tolist() == ([0, 0, 1, 0] if n else [0, 0, 0, 0])
    got = lm.policy_loss_backward(one, f.weights, x, a).double().cpu().numpy()
    assert (np.abs(got + adv / max(n, 1)) <= 4 * U * np.abs(adv) / max(n, 1)).all()
    for count, den in ((0, 0.0), (7, 1 / 7)):
        f = lm.policy_loss_forward(x, a, num_valid=count)
        assert abs(float(f.loss) + den * adv.sum()) <= 4 * U * size * n * den
        got = lm.policy_loss_backward(one, f.weights, x, a, num_valid=count).double().cpu().numpy()
        assert (np.abs(got + den * adv) <= 4 * U * np.abs(adv) * den).all()
        # a sequence mean over one sequence of all tokens
        f = lm.policy_loss_forward(x, a, reduction="sequence_mean", num_valid=count)
        assert abs(float(f.loss) + den * (adv.mean() if n else 0.0)) <= 4 * U * size * den


@pytest.mark.parametrize("n", [300, 30000])
@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
def test_policy_bad_numbers_in_ignored_places(n, reduction):
    rng, cu, targets, logp, old, ref_ = inputs(n, 6, "empty", 3)
    adv = f32(rng.standard_normal(n))
    _, ok = ref.counted(n, targets, cu)
    kw = dict(kl_weight=0.1, reduction=reduction)
    cu_, t = dev(cu, torch.int32), dev(targets, torch.int32)
    clean = [dev(v) for v in (logp, adv, old, ref_)]
    f = lm.policy_loss_forward(*clean, t, cu_, **kw)
    d = lm.policy_loss_backward(torch.ones(1, device="cuda"), f.weights, *clean, t, cu_, **kw)
    for bad in (float("nan"), float("inf"), -float("inf"), -3.4e38):
        dirty = [v.masked_fill(~dev(ok, torch.bool), bad) for v in clean]
        g = lm.policy_loss_forward(*dirty, t, cu_, **kw)
        e = lm.policy_loss_backward(torch.ones(1, device="cuda"), g.weights, *dirty, t, cu_, **kw)
        assert all(torch.equal(a, b) for a, b in zip(f, g)) and torch.equal(d, e)
    # in a place that counts it reaches the loss and its own gradient alone
    at = int(np.flatnonzero(ok)[len(np.flatnonzero(ok)) // 2])
    x = clean[0].clone()
    x[at] = float("nan")
    g = lm.policy_loss_forward(x, *clean[1:], t, cu_, **kw)
    e = lm.policy_loss_backward(torch.ones(1, device="cuda"), g.weights, x, *clean[1:], t, cu_, **kw)
    assert g.loss.isnan() and e[at].isnan() and int(e.isnan().sum()) == 1


def test_policy_border_in_64_bits():
    """Gaps one fp32 step on either side of log(1 + clip), where fp32 ratios tie."""
    edge = np.float32(np.log1p(0.2))
    gaps = np.array([np.nextafter(edge, np.float32(v)) for v in (0, 1)] + [edge], dtype=np.float32)
    low = np.float32(np.log1p(-0.2))
    downs = np.array([np.nextafter(low, np.float32(v)) for v in (-1, 0)] + [low], dtype=np.float32)
    logp = np.concatenate([gaps, downs]).astype(np.float64)   # old 0: the gap itself
    adv = np.array([1.0] * 3 + [-1.0] * 3)
    want = ref.policy(logp, adv, np.zeros(6), reduction="sum")
    x, a, o = dev(logp), dev(adv), torch.zeros(6, device="cuda")
    f = lm.policy_loss_forward(x, a, o, reduction="sum")
    got = lm.policy_loss_backward(torch.ones(1, device="cuda"), f.weights, x, a, o, reduction="sum").cpu().numpy()
    true_border = [g > np.log1p(0.2) for g in gaps.astype(np.float64)] + [g < np.log1p(-0.2) for g in downs.astype(np.float64)]
    assert [v == 0 for v in got] == true_border and len(set(true_border)) == 2
    assert abs(float(f.stats[1]) - sum(true_border) / 6) < 1e-7
    assert abs(float(f.loss) - want[0]) < 6 * 4 * U


@pytest.mark.parametrize("n", [0, 3, 700])
def test_more_sequences_than_a_workgroup_takes(n):
    """20,000 sequences over a few tokens, most of them empty."""
    rng = np.random.default_rng(n)
    sequences = 20000
    cu = np.sort(rng.integers(0, n + 1, sequences + 1))
    logp, old, adv = f32(-rng.random(n)), f32(-rng.random(n)), f32(rng.standard_normal(n))
    args = (dev(logp), dev(adv), dev(old), None, None, dev(cu, torch.int32))
    for reduction in ("mean", "sequence_mean"):
        want = ref.policy(logp, adv, old, None, None, cu, reduction=reduction)
        f = lm.policy_loss_forward(*args, reduction=reduction)
        got = lm.policy_loss_backward(torch.ones(1, device="cuda"), f.weights, *args, reduction=reduction)
        assert abs(float(f.loss) - want[0]) <= U * (want[3].sum() + 2 * abs(want[0])) * 1.01 + 1e-300
        assert (np.abs(got.double().cpu().numpy() - want[2]) <= U * (want[3] + 4 * np.abs(want[2])) * 1.01).all()
    want = ref.preference(logp, cu, None, None, average=True)
    f = lm.preference_loss_forward(args[0], args[5], average=True)
    got = lm.preference_loss_backward(torch.ones(1, device="cuda"), f.coef, n, args[5])
    assert abs(float(f.loss) - want[0]) <= 2 * U * want[0]
    # the slope's change with h: at most 1/4 of beta U (|s| + |s|), each |s| <= 1
    assert (np.abs(got.double().cpu().numpy() - want[2]) <= 2 * U * np.abs(want[2]) + 0.1 * 0.25 * 0.2 * U).all()


def test_policy_without_a_lower_border():
    """clip_low 1: a ratio is never below 0."""
    x, o, a = torch.tensor([-60.0, -1.0], device="cuda"), torch.zeros(2, device="cuda"), -torch.ones(2, device="cuda")
    f = lm.policy_loss_forward(x, a, o, clip_low=1.0, reduction="sum")
    got = lm.policy_loss_backward(torch.ones(1, device="cuda"), f.weights, x, a, o, clip_low=1.0, reduction="sum")
    assert float(f.stats[1]) == 0 and torch.allclose(got, x.exp(), rtol=1e-6, atol=0)


def test_autograd_captured():
    """Gradients through autograd in a graph, both losses behind a lookup and the log-probs."""
    n, hidden, vocab = 130, 128, 500
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    W = (torch.randn(vocab, hidden, generator=g, device="cuda") * 0.1).to(torch.bfloat16).requires_grad_()
    ids = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.randint(-50, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    cu = torch.tensor([0, 40, 70, 70, 130], dtype=torch.int32, device="cuda")
    adv, old = torch.randn(4, generator=g, device="cuda"), -torch.rand(n, generator=g, device="cuda")

    def step():
        logp = lm.logprob(lm.embedding(ids, W), W, targets, chunk=256)
        a, _ = lm.policy_loss(logp, adv, logp.detach() + 0.1, old, targets, cu, kl_weight=0.1)
        b, _ = lm.preference_loss(logp, cu, old, targets)
        return torch.autograd.grad(a + b, W)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (out,) = step()
    for rep in range(3):
        with torch.no_grad():
            W.normal_(0, 0.1)
        ids.copy_(torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step()[0]), rep


@pytest.mark.parametrize("x", [0.0, 1e-6, 1e-3, 0.1, 0.4999, 0.5001, 2.0, 30.0])
def test_k3_small_and_large(x):
    """Relative accuracy of the estimate, where the plain difference cancels."""
    for v in (x, -x):
        v = float(np.float32(v))
        f = lm.policy_loss_forward(dev(np.array([v])), dev(np.zeros(1)), None, dev(np.zeros(1)), kl_weight=1.0,
                                   reduction="sum")
        want = np.expm1(-np.float128(v)) + np.float128(v)
        # six steps of the series and a square; outside it terms up to 1 + e^-x + |x| against a sum of at least 0.1
        assert abs(float(f.loss) - float(want)) <= (20 * U if abs(v) <= 0.5 else 60 * U) * float(want), v


@pytest.mark.parametrize("n,pairs", [(2, 1), (3, 1), (500, 4), (8192, 2), (8193, 2), (20000, 900), (100003, 40)])
@pytest.mark.parametrize("kind", ["even", "empty", "skewed"])
@pytest.mark.parametrize("how", [dict(label_smoothing=0.2), dict(kind="hinge", beta=0.3, margin=0.2),
                                 dict(kind="squared", beta=0.5, average=True), dict(average=True, beta=2.0, margin=0.7),
                                 dict(num_pairs=11)])
def test_preference(n, pairs, kind, how):
    rng, cu, targets, logp, _, ref_ = inputs(n, 2 * pairs, kind, n + pairs)
    if n % 2:
        ref_ = None
    want = ref.preference(logp, cu, ref_, targets, **how)
    args = (dev(logp), dev(cu, torch.int32), dev(ref_), dev(targets, torch.int32))
    f = lm.preference_loss_forward(*args, **how)
    beta, average = how.get("beta", 0.1), how.get("average", False)
    # a token's difference is rounded once; sums are of 64 bits
    _, ok = ref.counted(n, targets, cu)
    gain = np.abs(logp - ref_) if ref_ is not None else np.abs(logp)
    size = np.array([gain[cu[s]:cu[s + 1]][ok[cu[s]:cu[s + 1]]].sum() /
                     (max(1, ok[cu[s]:cu[s + 1]].sum()) if average else 1) for s in range(2 * pairs)])
    dh = beta * U * (size[:pairs] + size[pairs:]) * 1.01 + 1e-15
    rewards = f.rewards.double().cpu().numpy()
    assert (np.abs(rewards - want[1]) <= beta * U * size * 1.01 + U * np.abs(want[1]) * 1.01 + 1e-15).all()
    # slopes: |l'| <= 1, or 2 |h - 1/2| / beta^2; their change: l'' <= 1/4, or 2 / beta^2; at the hinge's corner a step
    h = want[1][:pairs] - want[1][pairs:] - how.get("margin", 0.0)
    kind_ = how.get("kind", "sigmoid")
    if kind_ == "squared":
        first, second = 2 * (np.abs(h - 0.5) + dh) / beta ** 2, 2 / beta ** 2
    else:
        first, second = np.ones(pairs), 0.25
    if kind_ == "hinge":
        assert (np.abs(h - 1) > dh).all()
        second = 0.0
    den = how.get("num_pairs", pairs)
    assert abs(float(f.loss) - want[0]) <= (first * dh).sum() / den + 2 * U * abs(want[0]) + 1e-15
    grad = torch.tensor(0.5, device="cuda")
    got = lm.preference_loss_backward(grad, f.coef, n, args[1], args[3]).double().cpu().numpy()
    seq, _ = ref.counted(n, targets, cu)
    token_dh = np.where(seq >= 0, dh[np.clip(seq, 0, None) % pairs], 0.0)
    assert (np.abs(got - 0.5 * want[2]) <= 2 * U * np.abs(want[2]) + beta * second * token_dh / den).all()
    assert (got[~ok] == 0).all()
    again = lm.preference_loss_forward(*args, **how)
    assert all(torch.equal(a, b) for a, b in zip(f, again))


def test_preference_empty_buffer_and_far_margins():
    cu = torch.zeros(5, dtype=torch.int32, device="cuda")
    none = torch.empty(0, device="cuda")
    f = lm.preference_loss_forward(none, cu)
    assert abs(float(f.loss) - np.log(2)) < U and (f.rewards == 0).all()
    assert lm.preference_loss_backward(torch.ones(1, device="cuda"), f.coef, 0, cu).shape == (0,)
    # h = +-5000: the loss is 0 or 5000, its slope 0 or -1, nothing overflows
    logp = torch.tensor([0.0, -50000.0], device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for x, loss, slope in ((logp, 0.0, 0.0), (logp.flip(0), 5000.0, -1.0)):
        f = lm.preference_loss_forward(x, cu)
        g = lm.preference_loss_backward(torch.ones(1, device="cuda"), f.coef, 2, cu).tolist()
        assert abs(float(f.loss) - loss) < 1e-3 and g == pytest.approx([0.1 * slope, -0.1 * slope], rel=1e-6)
    x = torch.tensor([float("nan"), -1.0], device="cuda")
    for kind in ("sigmoid", "hinge", "squared"):
        assert lm.preference_loss_forward(x, cu, kind=kind).loss.isnan()
    # given counts: zero pairs
    f = lm.preference_loss_forward(logp, cu, num_pairs=0)
    assert float(f.loss) == 0 and (f.coef == 0).all()


def test_preference_ignored_places_and_bytes_behind():
    rng, cu, targets, logp, _, ref_ = inputs(20000, 10, "empty", 5)
    _, ok = ref.counted(20000, targets, cu)
    cu_, t = dev(cu, torch.int32), dev(targets, torch.int32)
    x, r = dev(logp), dev(ref_)
    f = lm.preference_loss_forward(x, cu_, r, t)
    for bad in (float("nan"), float("inf"), -3.4e38):
        y, q = (v.masked_fill(~dev(ok, torch.bool), bad) for v in (x, r))
        g = lm.preference_loss_forward(y, cu_, q, t)
        assert all(torch.equal(a, b) for a, b in zip(f, g))


def test_autograd():
    rng, cu, targets, logp, old, ref_ = inputs(3000, 8, "even", 9)
    t, cu_ = dev(targets, torch.int32), dev(cu, torch.int32)
    adv = dev(rng.standard_normal(8))
    x = dev(logp).requires_grad_()
    kw = dict(kl_weight=0.2, reduction="sequence_mean")
    loss, stats = lm.policy_loss(x, adv, dev(old), dev(ref_), t, cu_, **kw)
    (3.0 * loss).backward()
    f = lm.policy_loss_forward(x.detach(), adv, dev(old), dev(ref_), t, cu_, **kw)
    want = lm.policy_loss_backward(torch.tensor(3.0, device="cuda"), f.weights, x.detach(), adv, dev(old), dev(ref_), t,
                                   cu_, **kw)
    assert torch.equal(x.grad, want) and torch.equal(loss, f.loss) and not stats.requires_grad
    x.grad = None
    loss, rewards = lm.preference_loss(x, cu_, dev(ref_), t, average=True)
    loss.backward()
    f = lm.preference_loss_forward(x.detach(), cu_, dev(ref_), t, average=True)
    want = lm.preference_loss_backward(torch.ones(1, device="cuda"), f.coef, 3000, cu_, t)
    assert torch.equal(x.grad, want) and torch.equal(rewards, f.rewards) and not rewards.requires_grad
    # through both at once, and nothing from the statistics
    x.grad = None
    a, _ = lm.policy_loss(x, adv, cu_seqlens=cu_)
    b, _ = lm.preference_loss(x, cu_)
    (a + b).backward()
    assert x.grad.isfinite().all()
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad(lm.policy_loss(x, adv, cu_seqlens=cu_)[0], x, create_graph=True)
        g.sum().backward()


@pytest.mark.parametrize("n", [700, 40000])
def test_captured_and_replayed_with_eager_work_between(n):
    rng, cu, targets, logp, old, ref_ = inputs(n, 12, "empty", 21)
    x, o, r, a = dev(logp), dev(old), dev(ref_), dev(rng.standard_normal(n))
    t, cu_, one = dev(targets, torch.int32), dev(cu, torch.int32), torch.ones(1, device="cuda")

    def step():
        out = []
        for reduction in ("mean", "sequence_mean"):
            f = lm.policy_loss_forward(x, a, o, r, t, cu_, kl_weight=0.1, reduction=reduction)
            out += [*f, lm.policy_loss_backward(one, f.weights, x, a, o, r, t, cu_, kl_weight=0.1, reduction=reduction)]
        f = lm.preference_loss_forward(x, cu_, r, t)
        return out + [*f, lm.preference_loss_backward(one, f.coef, n, cu_, t)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        _, cu2, targets2, logp2, _, _ = inputs(n, 12, ["even", "empty", "skewed", "empty"][rep], 30 + rep)
        x.copy_(dev(logp2))
        t.copy_(dev(targets2, torch.int32))
        cu_.copy_(dev(cu2, torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, step()):
            assert torch.equal(p, q), rep


def test_refusals_of_the_helpers():
    x, cu = torch.zeros(6, device="cuda"), torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    t, one = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    for call in (lambda: lm.policy_loss(x.double(), x), lambda: lm.policy_loss(x, x[:3]), lambda: lm.policy_loss(x, x[:2]),
                 lambda: lm.policy_loss(x, x, x[:5]), lambda: lm.policy_loss(x, x, None, x.double()),
                 lambda: lm.policy_loss(x, x, targets=t[:5]), lambda: lm.policy_loss(x, x, targets=t.long()),
                 lambda: lm.policy_loss(x, x, cu_seqlens=cu.long()), lambda: lm.policy_loss(x, x, cu_seqlens=cu[:1]),
                 lambda: lm.policy_loss(x, x, kl_kind="k4"), lambda: lm.policy_loss(x, x, reduction="none"),
                 lambda: lm.policy_loss(x[::2], x[::2]),
                 lambda: lm.policy_loss(x[:2], x[:2], cu_seqlens=cu),   # 2 tokens, 2 sequences: whose advantages?
                 lambda: lm.policy_loss_backward(x, one, x, x), lambda: lm.policy_loss_backward(one, x, x, x),
                 lambda: lm.preference_loss(x, cu[:2]), lambda: lm.preference_loss(x, cu.repeat(2)),
                 lambda: lm.preference_loss(x, cu, x[:3]), lambda: lm.preference_loss(x, cu, kind="other"),
                 lambda: lm.preference_loss_backward(one, x[:3], 6, cu),
                 lambda: lm.preference_loss_backward(one, x[:2], 6, cu, t[:3])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lm.policy_loss(x, x, kl_weight=0.1), lambda: lm.policy_loss(x, x, clip_low=-1.0),
                 lambda: lm.policy_loss(x, x, dual_clip=0.5), lambda: lm.policy_loss(x, x, num_valid=-3),
                 lambda: lm.preference_loss(x, cu, beta=0.0), lambda: lm.preference_loss(x, cu, label_smoothing=0.7)):
        with pytest.raises(lm.LMHeadError):
            call()
