"""The losses on log-probabilities where they can go wrong: work in place on their
outputs, infinite numbers, weights of zero, the borders between launch shapes."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref
from test_gpu_token_losses import check_policy, dev, f32, inputs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ONE = dict(dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("kind", ["policy", "preference"])
@pytest.mark.parametrize("n", [300, 20000])
def test_work_in_place_on_the_outputs(kind, n):
    rng, cu, targets, logp, old, ref_ = inputs(n, 6, "even", 1)
    t, cu_ = dev(targets, torch.int32), dev(cu, torch.int32)
    x, adv = dev(logp).requires_grad_(), dev(rng.standard_normal(6))
    grads = []
    for how in range(3):
        if kind == "policy":
            loss, other = lm.policy_loss(x, adv, dev(old), dev(ref_), t, cu_, kl_weight=0.1, reduction="sequence_mean")
        else:
            loss, other = lm.preference_loss(x, cu_, dev(ref_), t)
        if how == 1:
            loss /= 4   # a power of two: the same bits, four times smaller
        elif how == 2:
            other.mul_(2)
            loss.detach().zero_()
        grads.append(torch.autograd.grad(loss, x)[0])
    assert torch.equal(grads[1] * 4, grads[0]) and torch.equal(grads[2], grads[0]) and (grads[0] != 0).any()
