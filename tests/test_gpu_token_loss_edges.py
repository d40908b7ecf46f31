"""The losses on log-probabilities where they can go wrong: work in place on their
outputs, infinite numbers, weights of zero, the borders between launch shapes."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref
from test_gpu_token_losses import dev, f32, inputs

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


@pytest.mark.parametrize("n", [300, 3000, 20000])
@pytest.mark.parametrize("reduction", ["mean", "sum", "sequence_mean"])
def test_a_reference_without_weight_takes_no_part(n, reduction):
    """A reference for the statistics alone, however far away: exp(ref - logp) passes
    fp32's range from 89 on."""
    rng, cu, targets, logp, old, ref_ = inputs(n, 6, "even", 2)
    _, ok = ref.counted(n, targets, cu)
    at = np.flatnonzero(ok)
    args = [dev(v) for v in (logp, rng.standard_normal(n), old)]
    t, cu_, one = dev(targets, torch.int32), dev(cu, torch.int32), torch.ones(1, **ONE)
    f = lm.policy_loss_forward(*args, None, t, cu_, reduction=reduction)
    want = lm.policy_loss_backward(one, f.weights, *args, None, t, cu_, reduction=reduction)
    assert f.loss.isfinite()
    for far in (logp + 100.0, np.full(n, np.inf), np.full(n, -np.inf), np.full(n, np.nan)):
        r = ref_.copy()
        r[at[::7]] = far[at[::7]]
        for kind in ("k1", "k2", "k3"):
            g = lm.policy_loss_forward(*args, dev(r), t, cu_, reduction=reduction, kl_kind=kind)
            d = lm.policy_loss_backward(one, g.weights, *args, dev(r), t, cu_, reduction=reduction, kl_kind=kind)
            assert torch.equal(g.loss, f.loss) and torch.equal(d, want) and torch.equal(g.stats[1:], f.stats[1:])
    # a reference at hand still gives its statistic
    g = lm.policy_loss_forward(*args, dev(ref_), t, cu_, reduction=reduction)
    x = (logp - ref_)[ok]
    k = np.expm1(-x) + x
    # as in check_policy: a token's estimate is off by its terms' roundings
    assert abs(float(g.stats[0]) - k.mean()) <= U * ((4 + 4 * np.abs(x) + 4 * np.exp(-x)).mean() + k.mean())


@pytest.mark.parametrize("n", [5, 3000, 20000])
def test_without_old_log_probs_a_ratio_is_one(n):
    """Whatever the log-prob: an infinite one too, as a masked token's. NaN stays NaN."""
    rng = np.random.default_rng(n)
    logp, adv = f32(-rng.random(n)), f32(rng.standard_normal(n))
    one = torch.ones(1, **ONE)
    clean = lm.policy_loss_forward(dev(logp), dev(adv))
    want = lm.policy_loss_backward(one, clean.weights, dev(logp), dev(adv))
    assert clean.stats.tolist() == [0, 0, 1, 0]
    for bad in (-np.inf, np.inf):
        x = logp.copy()
        x[::3] = bad
        f = lm.policy_loss_forward(dev(x), dev(adv))
        d = lm.policy_loss_backward(one, f.weights, dev(x), dev(adv))
        assert all(torch.equal(a, b) for a, b in zip(f, clean)) and torch.equal(d, want)
    x = logp.copy()
    x[3] = np.nan
    f = lm.policy_loss_forward(dev(x), dev(adv))
    d = lm.policy_loss_backward(one, f.weights, dev(x), dev(adv))
    assert f.loss.isnan() and d[3].isnan() and int(d.isnan().sum()) == 1


@pytest.mark.parametrize("n", [5, 3000, 20000])
@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
def test_a_given_count_of_zero_gives_zeros(n, reduction):
    """Also where a token's own term is infinite: a ratio past fp32's range, an
    estimate past it, a log-prob of -infinity or NaN."""
    rng = np.random.default_rng(n)
    logp, old, ref_ = f32(-rng.random(n)), f32(-rng.random(n)), f32(-rng.random(n))
    adv = -np.abs(f32(rng.standard_normal(n))) - 0.1
    old[0], ref_[1], logp[2], logp[3] = -200.0, 200.0, -np.inf, np.nan
    args = [dev(v) for v in (logp, adv, old, ref_)]
    kw = dict(kl_weight=0.1, reduction=reduction, num_valid=0)
    f = lm.policy_loss_forward(*args, **kw)
    d = lm.policy_loss_backward(torch.ones(1, **ONE), f.weights, *args, **kw)
    assert float(f.loss) == 0 and (f.weights == 0).all() and (d == 0).all()


@pytest.mark.parametrize("length,pairs", [(100, 1), (1000, 1), (700, 3), (20000, 1), (1500, 40), (10, 1100)])
def test_preference_differences_are_of_64_bits(length, pairs):
    """Tokens whose logp - ref an fp32 difference would round to 1, on the chosen side
    alone: what is lost there is all of h. Sums of `length` terms near 1 in 64 bits are
    within length^2 2^-53 of the true ones, and so is h by beta; then one rounding."""
    step = 2.0 ** -24
    logp = np.concatenate([np.full(pairs * length, -1.1 * step), np.zeros(pairs * length)])
    ref_ = np.concatenate([np.full(pairs * length, -1.0 - 2 * step), np.full(pairs * length, -1.0)])
    logp, ref_ = f32(logp), f32(ref_)
    cu = np.arange(2 * pairs + 1) * length
    beta = 0.5 / (length * 0.9 * step)   # h near 1/2
    assert (np.float32(logp) - np.float32(ref_) == 1).all()
    want = ref.preference(logp, cu, ref_, kind="hinge", beta=beta)
    args = (dev(logp), dev(cu, torch.int32), dev(ref_))
    f = lm.preference_loss_forward(*args, kind="hinge", beta=beta)
    assert 0.4 < want[0] < 0.6
    assert abs(float(f.loss) - want[0]) <= 2 * beta * length ** 2 * 2.0 ** -53 + U
    want = ref.preference(logp, cu, ref_, beta=beta)
    f = lm.preference_loss_forward(*args, beta=beta)
    got = lm.preference_loss_backward(torch.ones(1, **ONE), f.coef, len(logp), args[1]).double().cpu().numpy()
    # the slope moves by at most h's error / 4, then two roundings
    off = beta / pairs * (0.25 * 2 * beta * length ** 2 * 2.0 ** -53) + 2 * U * np.abs(want[2])
    assert (np.abs(got - want[2]) <= off).all()
