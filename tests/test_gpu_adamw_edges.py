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
