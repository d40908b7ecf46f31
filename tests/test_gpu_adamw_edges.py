"""The AdamW step where it can go wrong: NaN of every kind, vanishing second moments,
gradients that a program replaced."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref

pytestmark = pytest.mark.gpu

BF, F32, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.mark.parametrize("state", [F32, E8])
@pytest.mark.parametrize("seed", [None, 3])
@pytest.mark.parametrize("grad", [BF, F32])
def test_nan_of_any_bits_stays(state, seed, grad):
    """A NaN's fraction and sign are free: all ones too, which a sum of random bits would carry over."""
    bits = [0x7fc0, 0x7fff, 0xffff, 0xffc0, 0x7f81, 0xff81]
    n = 1280
    d = torch.full((n,), 0.5, device="cuda").to(grad)
    at = torch.arange(0, n, 16, device="cuda")
    if grad == BF:
        nans = torch.tensor([b - (1 << 16) if b > 0x7fff else b for b in bits], dtype=torch.int16, device="cuda").view(BF)
    else:
        full = [b << 16 | (b & 1) * 0xffff for b in bits]
        nans = torch.tensor([b - (1 << 32) if b >> 31 else b for b in full], dtype=torch.int32, device="cuda").view(F32)
    assert nans.isnan().all()
    d[at] = nans[torch.arange(len(at), device="cuda") % len(bits)]
    is_nan = torch.zeros(n, dtype=torch.bool, device="cuda")
    is_nan[at] = True
    p = torch.ones(n, device="cuda")
    s = lm.adamw_state(p, state)
    plan = lm.adamw_plan([p], [d], [s])
    for t in range(1, 4):
        lm.adamw_step(plan, t, 0.1, seed=seed)
        for x in (p, s.exp_avg.float(), s.exp_avg_sq.float()):
            assert torch.equal(x.isnan(), is_nan), t
        if t == 2:   # without them the states remember
            d.fill_(0.5)


@pytest.mark.parametrize("param", [BF, F32])
def test_second_moments_below_the_normal_numbers(param):
    """Gradients of 1e-20 .. 1e-18, whose v' lies among fp32's subnormals: with an eps
    far below them a step is still lr at most. v' is a multiple of 2^-149: its
    products and sum are off by half of one each beside the relative 2^-24."""
    n = 4000
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    d = torch.randn(n, generator=g, device="cuda").sign() * 10.0 ** (torch.rand(n, generator=g, device="cuda") * 2 - 20)
    p = torch.zeros(n, dtype=param, device="cuda")
    s = lm.adamw_state(p)
    h = dict(lr=0.5, beta1=0.9, beta2=0.97, eps=1e-36, weight_decay=0.0)
    plan = lm.adamw_plan([p], [d], [s])
    for t in (1, 2, 3):
        p0, d0, m0, v0 = (x.double().cpu().numpy() for x in (p, d, s.exp_avg, s.exp_avg_sq))
        lm.adamw_step(plan, t, **h)
        p1, m1, v1, den = ref.adamw(p0, d0, m0, v0, t, **h)
        assert (v1 < 2.0 ** -126).mean() > 0.5
        # as for normal numbers, the root halving v's error
        dm = U * (3 * 0.9 * np.abs(m0) + 4 * 0.1 * np.abs(d0)) * 1.01
        dv = U * (3 * 0.97 * v0 + 6 * 0.03 * d0 ** 2) * 1.01 + 2 * 2.0 ** -149
        quot = np.abs(m1) / den
        rel = dv / v1
        assert (rel < 0.01).all()
        dq = dm / den + quot * (rel / 2 * 1.02 + 9 * U)
        dp = 3 * U * np.abs(p0) + 0.5 / (1 - 0.9 ** t) * dq * 1.01 + (2.0 ** -8 if param == BF else U) * np.abs(p1)
        assert (np.abs(p.double().cpu().numpy() - p1) <= dp).all()
        assert (np.abs(s.exp_avg_sq.double().cpu().numpy() - v1) <= dv).all()
        d = d.neg_() if t == 1 else d


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_8_bit_states_of_vanishing_gradients(beta2):
    """Codes and scales bit for bit those of an elementwise program, where v' is subnormal."""
    n = 1 << 18
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    spread = torch.exp2(torch.rand(n, generator=g, device="cuda") * 6 - 66)
    p, d = torch.zeros(n, dtype=BF, device="cuda"), torch.randn(n, generator=g, device="cuda") * spread
    s = lm.adamw_state(p, E8)
    plan = lm.adamw_plan([p], [d], [s])
    m, v, ms, vs = (t.clone() if t.dtype != E8 else t.view(torch.uint8).clone().view(E8) for t in s)
    for t in (1, 2, 3):
        lm.adamw_step(plan, t, 0.01, 0.9, beta2, 1e-30)
        m1 = (m.float() * ms.repeat_interleave(128)) * 0.9 + d * (1.0 - 0.9)
        v1 = (v.float() * vs.repeat_interleave(128)).square() * beta2 + d.square() * (1.0 - beta2)
        assert float((v1 < 2.0 ** -126).float().mean()) > 0.1
        out = []
        for x, root in ((m1, False), (v1.double().sqrt().float(), True)):   # rounded once
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
        d.normal_(generator=g).mul_(spread)
