"""The AdamW step over many tensors against the plain 64-bit definition."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.97, eps=1e-6, weight_decay=0.1)


def f64(t):
    return t.double().cpu().numpy().ravel() if t.dtype != E8 else t.float().double().cpu().numpy().ravel()


def randn(g, shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def offset(t, by):
    """The same values at `by` elements from an aligned address."""
    flat = torch.empty(t.numel() + by, dtype=torch.uint8 if t.dtype == E8 else t.dtype, device="cuda")
    view = flat[by:].view(t.dtype).view(t.shape) if t.dtype == E8 else flat[by:].view(t.shape)
    view.copy_(t)
    return view


def make(g, shape, param, grad, state, copy, shift=0):
    n = int(np.prod(shape))
    move = (lambda t: offset(t, shift)) if shift else (lambda t: t)
    p, d = move(randn(g, shape, param)), move(randn(g, shape, grad, 0.1))
    m, v = randn(g, shape, std=0.05), randn(g, shape, std=0.3).exp() * 0.01
    c = move(torch.zeros(shape, dtype=BF, device="cuda")) if copy else None
    if state == F32:
        return p, d, lm.AdamWState(move(m), move(v)), c
    blocks = -(-n // 128)
    pad = lambda x: torch.nn.functional.pad(x.reshape(-1), (0, -n % 128)).view(blocks, 128)  # noqa: E731
    out = []
    for x in (m, v.sqrt()):
        s = (pad(x).abs().amax(1) / 448).clamp(min=1e-30)
        out.append((move((pad(x) / s[:, None]).to(E8).view(-1)[:n].view(shape)), s))
    return p, d, lm.AdamWState(out[0][0], out[1][0], out[0][1], out[1][1]), c


def before(item):
    p, d, s, c = item
    m, v = f64(s.exp_avg), f64(s.exp_avg_sq)
    if s.exp_avg_scale is not None:
        m = m * np.repeat(f64(s.exp_avg_scale), 128)[:m.size]
        v = (v * np.repeat(f64(s.exp_avg_sq_scale), 128)[:v.size]) ** 2
    return f64(p), f64(d), m, v


def check(item, was, step, hyper, scale=1.0):
    p, d, s, c = item
    p0, g0, m0, v0 = was
    g0 = g0 * scale
    h = dict(hyper)
    p1, m1, v1, den = ref.adamw(p0, g0, m0, v0, step, **h)
    b1, b2, lr = h["beta1"], h["beta2"], h["lr"]
    # roundings of 2^-24 each: the scaled gradient, a coefficient and a product
    # per term, one sum; 8-bit states first: value times scale, and its square
    e8 = s.exp_avg_scale is not None
    dm = U * ((3 + e8) * b1 * np.abs(m0) + 4 * (1 - b1) * np.abs(g0)) * 1.01
    dv = U * ((3 + 3 * e8) * b2 * v0 + 6 * (1 - b2) * g0 ** 2) * 1.01
    bc = 1 - b1 ** step
    # the root halves v's error; then its rounding, the factor, product, sum, quotient (up to 3), step size, fma
    quot = np.abs(m1) / den
    dq = dm / den + quot * (dv / (2 * np.maximum(v1, 1e-300)) + 9 * U)
    dp = U * 3 * np.abs(p0) + lr / bc * dq * 1.01
    if p.dtype == BF:
        dp = dp + 2.0 ** -8 * np.abs(p1)
    got = f64(p)
    assert (np.abs(got - p1) <= dp + 1e-37).all(), np.abs(got - p1).max()
    if c is not None:
        exact = torch.from_numpy(got).to(BF).double().numpy() if p.dtype == F32 else got
        assert np.array_equal(f64(c), exact)
    if not e8:
        assert (np.abs(f64(s.exp_avg) - m1) <= dm + 1e-45).all()
        assert (np.abs(f64(s.exp_avg_sq) - v1) <= dv + 1e-45).all()
        return
    for code, got_s, x, dx, root in ((s.exp_avg, s.exp_avg_scale, m1, dm, False),
                                     (s.exp_avg_sq, s.exp_avg_sq_scale, np.sqrt(v1), dv / (2 * np.sqrt(np.maximum(v1, 1e-300))), True)):
        want_s, each = ref.block_scale(x)
        dmax = np.zeros(want_s.size * 128)
        dmax[:x.size] = dx + U * np.abs(x)
        ds = dmax.reshape(-1, 128).max(1) / 448 + U * want_s
        assert (np.abs(f64(got_s) - want_s) <= ds * 1.01).all()
        each_got = np.repeat(f64(got_s), 128)[:x.size]
        q = f64(code)
        if root:
            assert (q[x > 1e-25] >= 2.0 ** -9).all()   # above zero stays above zero
            x = np.where((x > 0) & (x < 2.0 ** -9 * each_got), 2.0 ** -9 * each_got, x)
        # half a step: 2^-4 of the value, 2^-10 of the scale below the normal codes
        half = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * each_got)
        assert (np.abs(q * each_got - x) <= half * (1 + 4 * U) + dx + 2 * U * np.abs(x) + 448 * np.repeat(ds, 128)[:x.size]).all()


def run(items, step, hyper, scale=None):
    was = [before(i) for i in items]
    plan = lm.adamw_plan([i[0] for i in items], [i[1] for i in items], [i[2] for i in items], [i[3] for i in items])
    gs = None if scale is None else torch.tensor([scale], device="cuda")
    lm.adamw_step(plan, step, grad_scale=gs, **hyper)
    for i, w in zip(items, was):
        check(i, w, step, hyper, 1.0 if scale is None else float(np.float32(scale)))
    return plan


SHAPES = [(1,), (7,), (128,), (129, 3), (4095,), (4096,), (4097,), (33, 1000)]


@pytest.mark.parametrize("state", [F32, E8])
@pytest.mark.parametrize("param", [BF, F32])
@pytest.mark.parametrize("grad", [BF, F32])
@pytest.mark.parametrize("step", [1, 40])
def test_step(state, param, grad, step):
    g = torch.Generator(device="cuda")
    g.manual_seed(step)
    items = [make(g, shape, param, grad, state, i % 2 == 0) for i, shape in enumerate(SHAPES)]
    run(items, step, HYPER)
    run(items, step + 1, dict(HYPER, weight_decay=0.0, beta1=0.0), scale=0.37)


@pytest.mark.parametrize("state", [F32, E8])
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_tensors_at_any_element(state, shift):
    """Not 16-byte aligned, each buffer alone; elements before and behind stay."""
    g = torch.Generator(device="cuda")
    g.manual_seed(shift)
    for n in (5, 128, 1000, 5001):
        for param, grad in ((BF, F32), (F32, BF)):
            run([make(g, (n,), param, grad, state, True, shift)], 3, HYPER)
    # two tensors side by side in one buffer, a gap of three elements that keep their values
    flat = [torch.full((2003,), 7.0, device="cuda") for _ in range(4)]
    cut = (slice(0, 1000), slice(1003, 2003))
    items = [(flat[0][c], flat[1][c], lm.AdamWState(flat[2][c], flat[3][c]), None) for c in cut]
    run(items, 2, HYPER)
    assert all((f[1000:1003] == 7.0).all() for f in flat)


def test_mixed_tensors_over_several_launches():
    """130 tensors, types mixed in one plan, some of them empty."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rng = np.random.default_rng(4)
    kinds = [(p, d, s) for p in (BF, F32) for d in (BF, F32) for s in (F32, E8)]
    items = []
    for i in range(130):
        n = int(rng.integers(1, 9000)) if i % 11 else 0
        items.append(make(g, (n,), *kinds[i % 8], i % 3 == 0))
    run(items, 7, HYPER)


def test_a_table_gives_the_same_bits():
    """49 to 200 tensors: one launch from the table, or several without; at random rounding too."""
    rng = np.random.default_rng(12)
    for count in (49, 64, 65, 200):
        sizes = [int(rng.integers(0, 7000)) if i % 7 else 0 for i in range(count)]
        outs = []
        for table in (True, False):
            g = torch.Generator(device="cuda")
            g.manual_seed(count)
            items = [make(g, (n,), BF, BF, E8 if i % 3 else F32, False) for i, n in enumerate(sizes)]
            plan = lm.adamw_plan(*[[i[k] for i in items] for k in range(3)])
            assert plan.table is not None
            if not table:
                plan.table = None
            lm.adamw_step(plan, 3, 0.01)
            lm.adamw_step(plan, 4, 0.01, seed=5)
            outs.append([t.float() for i in items for t in (i[0], *i[2]) if t is not None])
        assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_one_tensor_of_many_chunks():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    for state in (F32, E8):
        run([make(g, (3_000_001,), BF, BF, state, False)], 2, HYPER)


def test_element_offsets_past_4_gib():
    """An fp32 tensor of 2^30 + 200 elements: its last ones, and its first."""
    n = 2 ** 30 + 200
    p, d = torch.ones(n, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    s = lm.AdamWState(torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"))
    d[0], d[-1] = 2.0, -4.0
    lm.adamw_step(lm.adamw_plan([p], [d], [s]), 1, 0.5, 0.9, 0.99, 1e-8, 0.0)
    # the first step moves by lr against the sign of the gradient
    assert abs(float(p[0]) - 0.5) < 1e-6 and abs(float(p[-1]) - 1.5) < 1e-6
    assert int((p != 1.0).sum()) == 2 and abs(float(s.exp_avg[-1]) + 0.4) < 1e-6


@pytest.mark.parametrize("state", [F32, E8])
def test_bad_numbers_and_vanishing_ones(state):
    """NaN stays in its element; an infinite gradient leaves no finite value of
    its 8-bit block behind; zeros do not move; tiny gradients stay above zero."""
    n = 400
    p = torch.ones(n, device="cuda")
    d = torch.full((n,), 0.5, device="cuda")
    s = lm.adamw_state(p, state)
    d[5], d[200:256] = float("nan"), 0.0
    plan = lm.adamw_plan([p], [d], [s])
    lm.adamw_step(plan, 1, 0.1)
    assert p[5].isnan() and int(p.isnan().sum()) == 1 and (p[200:256] == 1.0).all()
    assert int(s.exp_avg.float().isnan().sum()) == 1 and int(s.exp_avg_sq.float().isnan().sum()) == 1
    assert (s.exp_avg_sq.float()[200:256] == 0).all()
    if state == E8:
        assert s.exp_avg_scale.isfinite().all()
        p, d = torch.ones(256, device="cuda"), torch.full((256,), 1e-6, device="cuda")
        s = lm.adamw_state(p, state)
        d[3], d[130:] = 1e4, 0.0
        lm.adamw_step(lm.adamw_plan([p], [d], [s]), 1, 0.1)
        q = s.exp_avg_sq.float()
        assert (q[:128] >= 2.0 ** -9).all() and q[128] > 0 and (q[130:] == 0).all()
        # a step without a gradient moves nothing far: m' is zero or its denominator is not
        d.zero_()
        was = p.clone()
        lm.adamw_step(lm.adamw_plan([p], [d], [s]), 2, 0.1)
        assert ((p - was).abs() <= 0.11).all()
        d[3] = float("inf")
        lm.adamw_step(lm.adamw_plan([p], [d], [s]), 3, 0.1)
        assert s.exp_avg_scale[0].isinf() and s.exp_avg_scale[1].isfinite()


def test_all_zero_gradients_keep_zero_states():
    p = torch.ones(300, dtype=BF, device="cuda")
    d = torch.zeros(300, dtype=BF, device="cuda")
    for state in (F32, E8):
        s = lm.adamw_state(p, state)
        for t in (1, 2):
            lm.adamw_step(lm.adamw_plan([p], [d], [s]), t, 0.1)
        assert (p == 1).all() and (s.exp_avg.float() == 0).all() and (s.exp_avg_sq.float() == 0).all()


def test_step_rate_and_scale_on_the_device():
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    a = [make(g, (5000,), BF, BF, F32, False), make(g, (300,), F32, F32, E8, True)]
    b = [tuple(t.clone() if isinstance(t, torch.Tensor) else t if t is None else
               lm.AdamWState(*[u.clone() if u is not None else None for u in t]) for t in i) for i in a]
    plans = [lm.adamw_plan(*[[i[k] for i in items] for k in range(4)]) for items in (a, b)]
    step = torch.tensor([9], dtype=torch.int32, device="cuda")
    lr = torch.tensor(0.01, device="cuda")
    h = {k: v for k, v in HYPER.items() if k != "lr"}
    lm.adamw_step(plans[0], 9, float(lr), **h)
    lm.adamw_step(plans[1], step, lr, **h)
    for i, j in zip(a, b):
        # the powers of beta are taken by two libraries: factors may differ by a rounding
        assert torch.allclose(i[0].float(), j[0].float(), rtol=2.0 ** -7 if i[0].dtype == BF else 4 * U, atol=1e-7)
        assert torch.equal(i[2].exp_avg.float(), j[2].exp_avg.float())
    step.fill_(0)   # below 1 counts as 1
    was = [before(i) for i in b]
    lm.adamw_step(plans[1], step, lr, **h)
    for i, w in zip(b, was):
        check(i, w, 1, dict(h, lr=float(lr)))


def test_captured_and_replayed_with_eager_work_between():
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    items = [make(g, (n,), BF, BF, s, False) for n, s in ((4097, F32), (1000, E8), (64, F32))]
    plan = lm.adamw_plan(*[[i[k] for i in items] for k in range(3)])
    step, lr = torch.ones(1, dtype=torch.int32, device="cuda"), torch.full((1,), 0.01, device="cuda")
    lm.adamw_step(plan, step, lr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.adamw_step(plan, step, lr)
        step += 1
    for rep in range(4):
        for i in items:
            i[1].normal_()
        lr.fill_(0.01 / (1 + rep))
        was = [before(i) for i in items]
        t = int(step)
        graph.replay()
        torch.cuda.synchronize()
        assert int(step) == t + 1
        for i, w in zip(items, was):
            check(i, w, t, dict(lr=float(lr), beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0))


def test_repeats_bit_for_bit_and_on_another_stream():
    outs = []
    for rep in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(8)
        items = [make(g, (9001,), BF, BF, E8, True), make(g, (70001,), F32, BF, F32, False)]
        plan = lm.adamw_plan(*[[i[k] for i in items] for k in range(4)])
        torch.cuda.synchronize()
        stream = torch.cuda.Stream() if rep else torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            for t in range(1, 4):
                lm.adamw_step(plan, t, 0.01)
        torch.cuda.synchronize()
        outs.append([t.float().clone() for i in items for t in (i[0], *i[2]) if t is not None])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


@pytest.mark.parametrize("step,beta2", [(1, 0.95), (3, 0.999), (1000, 0.95)])
def test_8_bit_states_are_those_of_an_elementwise_program(step, beta2):
    """Codes and scales bit for bit over three steps: a code's step more or less
    would be the next step's scale where it is its block's largest."""
    g = torch.Generator(device="cuda")
    g.manual_seed(step)
    n = 1 << 22
    p, d, s, _ = make(g, (n,), BF, BF, E8, False)
    m, v, ms, vs = (t.clone() if t.dtype != E8 else t.view(torch.uint8).clone().view(E8) for t in s)
    plan = lm.adamw_plan([p], [d], [s])
    for t in range(step, step + 3):
        lm.adamw_step(plan, t, 0.01, 0.9, beta2)
        m1 = (m.float() * ms.repeat_interleave(128)) * 0.9 + d.float() * (1.0 - 0.9)
        v1 = (v.float() * vs.repeat_interleave(128)).square() * beta2 + d.float().square() * (1.0 - beta2)
        out = []
        for x, root in ((m1, False), (v1.sqrt(), True)):
            b = x.view(-1, 128)
            scale = b.abs().amax(1) * torch.tensor(1.0 / 448.0, device="cuda")
            y = b / scale[:, None]
            if root:
                y = torch.where(b > 0, y.clamp(min=2.0 ** -9), 0.0)
            out += [y.to(E8).view(-1), scale]
        m, ms, v, vs = out
        assert torch.equal(s.exp_avg_scale, ms) and torch.equal(s.exp_avg_sq_scale, vs)
        assert torch.equal(s.exp_avg.view(torch.uint8), m.view(torch.uint8))
        assert torch.equal(s.exp_avg_sq.view(torch.uint8), v.view(torch.uint8))
        d.normal_(generator=g)


def scramble(x):
    x = x & 0xffffffff
    x = (x ^ (x >> 16)) * 0x9e3779b9 & 0xffffffff
    x = (x ^ (x >> 15)) * 0xb7e15163 & 0xffffffff
    return x ^ (x >> 16)


@pytest.mark.parametrize("param,grad", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_random_rounding_is_the_documented_one(param, grad):
    """The codes from seed, step, place and element; parameters and scales as without."""
    g = torch.Generator(device="cuda")
    g.manual_seed(10)
    items = [make(g, (n,), param, grad, E8, False) for n in (300, 5000)]
    d = [items[1][1].clone(), items[1][1]]
    d[1][::7] *= 1e-4   # codes below the normal ones too
    twin = [(p.clone(), d, lm.AdamWState(*[(t.view(torch.uint8) if t.dtype == E8 else t).clone().view(t.dtype) for t in s]), c)
            for p, d, s, c in items]
    exact = [(p.clone(), d, lm.AdamWState((s[0].float() * s[2].repeat_interleave(128)[:s[0].numel()]),
                                          (s[1].float() * s[3].repeat_interleave(128)[:s[0].numel()]).square()), c)
             for p, d, s, c in items]
    plans = [lm.adamw_plan(*[[i[k] for i in group] for k in range(4)]) for group in (items, twin, exact)]
    lm.adamw_step(plans[0], 5, seed=77, **HYPER)
    for plan in plans[1:]:
        lm.adamw_step(plan, 5, **HYPER)
    ups = []
    for place, (a, b, e) in enumerate(zip(items, twin, exact)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2][2], b[2][2]) and torch.equal(a[2][3], b[2][3])
        n = a[0].numel()
        mix = scramble(77 + scramble(5 + scramble(place)))
        noise = scramble(np.arange(n, dtype=np.uint64) ^ np.uint64(mix))
        for code, scale, value, bits in ((a[2][0], a[2][2], f64(e[2][0]), noise & 0xffff),
                                         (a[2][1], a[2][3], np.sqrt(f64(e[2][1])), noise >> np.uint64(16))):
            y = np.abs(value) / np.repeat(f64(scale), 128)[:n]
            if code is a[2][1]:
                y = np.where((value > 0) & (y < 2.0 ** -9), 2.0 ** -9, y)
            step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(y, 1e-30))) - 3), 2.0 ** -9)
            want = np.floor(y / step + bits / 65536.0) * step
            got = np.abs(f64(code))
            # y and the fp32 state's are equal but for a few roundings: where the sum lies next to a code either will do
            near = np.abs((y / step + bits / 65536.0) % 1.0 - 0.5) > 0.5 - 64 * U * np.maximum(1, y / step) - 2.0 ** -19
            assert np.array_equal(got[~near], want[~near]) and near.mean() < 0.01
            assert (np.abs(got - want)[near] <= 2 * step[near]).all()
            ups.append((got > y).mean())
    assert 0.2 < np.mean(ups) < 0.8
    # another seed, step or place gives other codes; the same ones give the same
    def codes(step, seed):
        fresh = [(p.clone(), d, lm.AdamWState(*[(t.view(torch.uint8) if t.dtype == E8 else t).clone().view(t.dtype) for t in s]), None)
                 for p, d, s, _ in twin]
        lm.adamw_step(lm.adamw_plan(*[[i[k] for i in fresh] for k in range(4)]), step, seed=seed, **HYPER)
        return fresh[1][2][1].float()
    assert torch.equal(codes(5, 1), codes(5, 1))
    assert not torch.equal(codes(5, 1), codes(5, 2))


def test_random_rounding_takes_the_step_from_the_device():
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    a = make(g, (3000,), BF, BF, E8, False)
    b = (a[0].clone(), a[1], lm.AdamWState(*[(t.view(torch.uint8) if t.dtype == E8 else t).clone().view(t.dtype) for t in a[2]]), None)
    plans = [lm.adamw_plan([i[0]], [i[1]], [i[2]]) for i in (a, b)]
    lm.adamw_step(plans[0], 12, 0.01, seed=3)
    lm.adamw_step(plans[1], torch.tensor([12], dtype=torch.int32, device="cuda"), 0.01, seed=3)
    assert all(torch.equal(x.float(), y.float()) for x, y in zip(a[2], b[2]))


def test_8_bit_states_with_random_rounding_follow_fp32_ones():
    """300 steps on gradients of fixed spread: sqrt(v) is the fp32 state's on
    average. Its rounding noise: a step of at most 2^-3 of the value, taken with
    the probability p of the rest, has the variance p (1 - p) 2^-6 <= 2^-8; the
    state forgets at a rate of 0.005 a step, but what moves it a step is only its
    drift of at most about 0.005 2 / 2^-4, so the variance is at most about
    0.16 2^-6 / (2 0.005) = 0.25: a spread below 0.5, and the mean of 8192 of them
    is within 5 0.5 / 90 < 0.03 of 1, but for the root's curvature (E s^2 >= (E
    s)^2: up to half the variance)."""
    n = 8192
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    sigma = torch.exp2(torch.rand(n, generator=g, device="cuda") * 4 - 8)
    ps = [torch.zeros(n, device="cuda") for _ in range(2)]
    d = torch.zeros(n, device="cuda")
    states = [lm.adamw_state(ps[0]), lm.adamw_state(ps[1], E8)]
    plans = [lm.adamw_plan([p], [d], [s]) for p, s in zip(ps, states)]
    for t in range(1, 301):
        d.copy_(torch.randn(n, generator=g, device="cuda") * sigma)
        lm.adamw_step(plans[0], t, 1e-3, 0.9, 0.99)
        lm.adamw_step(plans[1], t, 1e-3, 0.9, 0.99, seed=1)
    root = states[0].exp_avg_sq.sqrt()
    got = states[1].exp_avg_sq.float() * states[1].exp_avg_sq_scale.repeat_interleave(128)
    ratio = (got / root).double()
    assert 0.85 < float(ratio.mean()) < 1.03 and float(ratio.std()) < 0.5
    # without gradients it falls as fp32 states do, by 0.99^100 in v, where nearest rounding would hold single ones up
    d.zero_()
    d[::128] = sigma[::128]   # the block's scale stays up
    for t in range(301, 401):
        for plan, seed in zip(plans, (None, 1)):
            lm.adamw_step(plan, t, 1e-3, 0.9, 0.99, seed=seed)
    got2 = states[1].exp_avg_sq.float() * states[1].exp_avg_sq_scale.repeat_interleave(128)
    rest = torch.arange(n, device="cuda") % 128 != 0
    fell = (got2[rest].double().sum() / got[rest].double().sum()).item()
    assert abs(fell - 0.99 ** 50) < 0.1 * 0.99 ** 50


def test_plans_refuse():
    p = torch.zeros(256, device="cuda")
    s = lm.adamw_state(p)
    e = lm.adamw_state(p, E8)
    d = torch.zeros_like(p)
    bad = [
        ([p], [d[:128]], [s]), ([p], [d.double()], [s]), ([p.half()], [d], [s]), ([p], [d], [lm.AdamWState(s[0], e[1])]),
        ([p], [d], [lm.AdamWState(e[0], e[1])]), ([p], [d], [lm.AdamWState(s[0], s[1], e[2], e[3])]),
        ([p], [d], [lm.AdamWState(e[0], e[1], e[2][:1], e[3])]), ([p], [d.cpu()], [s]), ([p], [None], [s]),
        ([p.view(16, 16).t()], [d.view(16, 16)], [lm.AdamWState(s[0].view(16, 16), s[1].view(16, 16))]),
        ([p, p], [d, d.clone()], [s, lm.adamw_state(p)]),   # one parameter twice
        ([p], [p], [s]), ([p], [d], [lm.AdamWState(s[0], s[0])]),
        ([p[:200], p[100:]], [d[:200], d[56:].clone()[:156]], [lm.adamw_state(p[:200]), lm.adamw_state(p[100:])]),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            lm.adamw_plan(*args)
    with pytest.raises(ValueError):
        lm.adamw_plan([p], [d], [s], [p.clone()])   # a copy is bf16
    plan = lm.adamw_plan([p], [d], [s])
    for kw in (dict(step=0, lr=0.1), dict(step=1, lr=float("nan")), dict(step=1, lr=0.1, eps=0.0),
               dict(step=1, lr=0.1, beta1=1.0), dict(step=1, lr=0.1, weight_decay=-1.0)):
        with pytest.raises(lm.LMHeadError):
            lm.adamw_step(plan, **kw)
    for kw in (dict(step=torch.ones(1, device="cuda"), lr=0.1), dict(step=1, lr=torch.ones(2, device="cuda")),
               dict(step=1, lr=torch.ones(1)), dict(step=1, lr=0.1, grad_scale=torch.ones(1, dtype=BF, device="cuda"))):
        with pytest.raises(ValueError):
            lm.adamw_step(plan, **kw)
    assert (p == 0).all()


def test_a_plan_keeps_its_storages():
    """Tensors that the caller drops stay alive in the plan."""
    p = torch.ones(1000, device="cuda")
    d = torch.ones_like(p)
    plan = lm.adamw_plan([p], [d], [lm.adamw_state(p)])
    del d
    junk = [torch.full((1000,), float("nan"), device="cuda") for _ in range(8)]
    lm.adamw_step(plan, 1, 0.5)
    assert abs(float(p[0]) - 0.5) < 1e-5 and len(junk) == 8
