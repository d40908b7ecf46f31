"""Refusals and sizes of include/lmhead_train.h, on the host: every call here
fails validation (fake addresses are never dereferenced) or, with valid
arguments and no device, ends in LMHEAD_ERR_DEVICE. Also the plain definitions
the GPU tests compare with, against differences, and the binding's own checks."""
import contextlib
import ctypes
import inspect
import os
import re

import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
BIG = 1 << 50
A, S, AL, W = lm.LMHEAD_ERR_ARG, lm.LMHEAD_ERR_SHAPE, lm.LMHEAD_ERR_ALIGN, lm.LMHEAD_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def test_library_exports_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lmhead_train.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lmhead_[a-z_0-9]+)\s*\(", text)))
    assert names == ["lmhead_adamw_step", "lmhead_adamw_table", "lmhead_adamw_table_size", "lmhead_embedding_bwd", "lmhead_embedding_bwd_workspace_size",
                     "lmhead_embedding_fwd", "lmhead_policy_loss_bwd", "lmhead_policy_loss_fwd",
                     "lmhead_policy_loss_workspace_size", "lmhead_preference_loss_bwd",
                     "lmhead_preference_loss_fwd", "lmhead_preference_loss_workspace_size"]
    L = ctypes.CDLL(lm.LIB_PATH)
    for name in names:
        assert hasattr(L, name) and hasattr(lm, name), name


def emb(**kw):
    d = dict(n=4, vocab=1000, hidden=256, scale=1.0, weight_dtype=0, out_dtype=0, accumulate=0)
    d.update(kw)
    return lm.lmhead_embedding(*d.values())


def test_embedding_refusals():
    F = FAKE
    ok = dict(ids=F, weight=F, scale=None, out=F, ws=None, bytes=0, stream=0)

    def call(p, **kw):
        return lm.lmhead_embedding_fwd(p, *{**ok, **kw}.values())
    for bad in (dict(weight_dtype=3), dict(weight_dtype=-1), dict(out_dtype=2), dict(accumulate=2), dict(scale=NAN),
                dict(scale=INF)):
        assert call(emb(**bad)) == A, bad
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(hidden=0),
                dict(hidden=100), dict(hidden=65600)):
        assert call(emb(**bad)) == S, bad
    assert call(emb(hidden=192, weight_dtype=2), scale=F) == S   # 8-bit: whole blocks
    for name in ("ids", "weight", "out"):
        assert call(emb(), **{name: None}) == A, name
        assert call(emb(), **{name: F + (2 if name == "ids" else 8)}) == AL, name
    assert call(emb(), scale=F) == A and call(emb(weight_dtype=2)) == A   # scales and 8-bit go together
    assert call(emb(weight_dtype=2), scale=F + 2) == AL
    assert call(emb(), ws=F + 16, bytes=256) == AL and call(emb(), ws=F, bytes=255) == W


def test_embedding_backward_refusals():
    F, size = FAKE, lm.lmhead_embedding_bwd_workspace_size
    ok = dict(ids=F, dout=F, dweight=F, ws=F, bytes=BIG, stream=0)

    def call(p, **kw):
        return lm.lmhead_embedding_bwd(p, *{**ok, **kw}.values())
    for bad in (dict(weight_dtype=2), dict(out_dtype=2), dict(accumulate=-1), dict(scale=INF)):
        assert call(emb(**bad)) == A and size(emb(**bad)) == 0, bad
    for bad in (dict(n=-1), dict(hidden=100), dict(vocab=0), dict(n=(1 << 26) + 1), dict(vocab=(1 << 28) + 1),
                dict(n=1 << 26, hidden=8192)):
        assert call(emb(**bad)) == S and size(emb(**bad)) == 0, bad
    for name in ("ids", "dout", "dweight", "ws"):
        assert call(emb(), **{name: None}) == A, name
        assert call(emb(), **{name: F + 2}) == AL, name
    assert call(emb(n=0), ids=None, dout=None, dweight=None) == A   # an empty call still writes zeros
    assert call(emb(), bytes=size(emb()) - 1) == W
    # four regions by tokens, and two rows of partial sums for each window of 16
    assert size(emb(n=16)) == 4 * 256 and size(emb(n=0)) == 256
    assert size(emb(n=17)) == 4 * 256 + 2 * 2 * 256 * 4


def pol(**kw):
    d = dict(n=4, sequences=2, num_valid=-1, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_weight=0.1, kl_kind=3,
             reduction=0, advantage_per_sequence=0, reserved=0)
    d.update(kw)
    return lm.lmhead_policy_problem(*d.values())


BAD_POLICY = (dict(reserved=1), dict(num_valid=-2), dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=NAN),
              dict(clip_high=-0.1), dict(clip_high=NAN), dict(clip_high=INF), dict(clip_high=1e300), dict(dual_clip=1.0),
              dict(dual_clip=-1.0), dict(dual_clip=NAN), dict(dual_clip=INF), dict(kl_weight=NAN), dict(kl_weight=INF),
              dict(kl_kind=0), dict(kl_kind=4), dict(reduction=-1), dict(reduction=3),
              dict(advantage_per_sequence=2), dict(advantage_per_sequence=1, sequences=0))


def test_policy_refusals():
    F, size = FAKE, lm.lmhead_policy_loss_workspace_size
    fwd = dict(logp=F, old=F, ref=F, adv=F, targets=F, cu=F, loss=F, stats=F, weights=F, ws=F, bytes=BIG, stream=0)
    bwd = dict(grad=F, weights=F, logp=F, old=F, ref=F, adv=F, targets=F, cu=F, dlogp=F, stream=0)

    def forward(p, **kw):
        return lm.lmhead_policy_loss_fwd(p, *{**fwd, **kw}.values())

    def backward(p, **kw):
        return lm.lmhead_policy_loss_bwd(p, *{**bwd, **kw}.values())
    for bad in BAD_POLICY:
        assert forward(pol(**bad)) == A and backward(pol(**bad)) == A and size(pol(**bad)) == 0, bad
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(sequences=-1), dict(sequences=(1 << 24) + 1)):
        assert forward(pol(**bad)) == S and backward(pol(**bad)) == S and size(pol(**bad)) == 0, bad
    for f, given in ((forward, fwd), (backward, bwd)):
        for name in ("logp", "adv", "ref", "cu"):   # ref: the KL's weight is not 0; cu: two sequences
            assert f(pol(), **{name: None}) == A, name
        assert f(pol(sequences=0)) == A             # cu_seqlens without sequences
        for name in given:
            if name not in ("ws", "bytes", "stream"):
                assert f(pol(), **{name: F + 2}) == AL, name
    for name in ("loss", "weights", "ws"):
        assert forward(pol(), **{name: None}) == A, name
    for name in ("grad", "weights", "dlogp"):
        assert backward(pol(), **{name: None}) == A, name
    assert forward(pol(), ws=F + 64) == AL and forward(pol(), bytes=0) == W
    # one launch needs none; above 4096 tokens six sums a tile of 1024, and with sequence means their parts
    assert size(pol(n=4096)) == 256 and size(pol(n=6 * 1024)) == 512
    assert size(pol(n=6 * 1024, reduction=2)) == 512 + 2 * 256
    assert size(pol(n=0, sequences=8193, reduction=2)) == 256 + 131328 + 65792   # 8194 parts of 16 bytes, 8193 means


def pref(**kw):
    d = dict(n=4, pairs=2, num_pairs=-1, beta=0.1, margin=0.0, label_smoothing=0.0, kind=0, average=0)
    d.update(kw)
    return lm.lmhead_preference_problem(*d.values())


def test_preference_refusals():
    F, size = FAKE, lm.lmhead_preference_loss_workspace_size
    fwd = dict(logp=F, ref=F, targets=F, cu=F, loss=F, rewards=F, coef=F, ws=F, bytes=BIG, stream=0)
    bwd = dict(grad=F, coef=F, targets=F, cu=F, dlogp=F, stream=0)

    def forward(p, **kw):
        return lm.lmhead_preference_loss_fwd(p, *{**fwd, **kw}.values())

    def backward(p, **kw):
        return lm.lmhead_preference_loss_bwd(p, *{**bwd, **kw}.values())
    for bad in (dict(num_pairs=-2), dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(beta=INF), dict(beta=1e-60),
                dict(margin=NAN), dict(margin=INF), dict(label_smoothing=-0.1), dict(label_smoothing=0.6),
                dict(label_smoothing=NAN), dict(label_smoothing=0.1, kind=1), dict(kind=3), dict(kind=-1),
                dict(average=2)):
        assert forward(pref(**bad)) == A and backward(pref(**bad)) == A and size(pref(**bad)) == 0, bad
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(pairs=0), dict(pairs=(1 << 23) + 1)):
        assert forward(pref(**bad)) == S and backward(pref(**bad)) == S and size(pref(**bad)) == 0, bad
    for name in ("logp", "cu", "loss", "coef", "ws"):
        assert forward(pref(), **{name: None}) == A, name
    for name in ("grad", "coef", "cu", "dlogp"):
        assert backward(pref(), **{name: None}) == A, name
    for f, given in ((forward, fwd), (backward, bwd)):
        for name in given:
            if name not in ("ws", "bytes", "stream"):
                assert f(pref(), **{name: F + 2}) == AL, name
    assert forward(pref(), ws=F + 64) == AL and forward(pref(), bytes=0) == W


def adam(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, device_step=None, device_lr=None,
             grad_scale=None, stochastic=0, seed=0)
    d.update(kw)
    return lm.lmhead_adamw(*d.values())


def tensor(**kw):
    d = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scale=None, exp_avg_sq_scale=None, copy=None,
             numel=100, param_dtype=0, grad_dtype=0, state_dtype=1, reserved=0)
    d.update(kw)
    return lm.lmhead_adamw_tensor(*d.values())


def test_adamw_refusals():
    f, F = lm.lmhead_adamw_step, FAKE

    def call(p, *tensors):
        return f(p, (lm.lmhead_adamw_tensor * len(tensors))(*tensors), len(tensors), None, 0)
    for bad in (dict(lr=NAN), dict(lr=INF), dict(weight_decay=-0.1), dict(weight_decay=NAN), dict(beta1=1.0),
                dict(beta1=-0.1), dict(beta1=NAN), dict(beta2=1.0), dict(beta2=1 - 1e-12), dict(beta2=NAN), dict(eps=0.0),
                dict(eps=1e-45), dict(eps=NAN), dict(eps=INF), dict(step=0), dict(step=-1),
                dict(stochastic=2)):
        assert call(adam(**bad), tensor()) == A, bad
    for name in ("device_step", "device_lr", "grad_scale"):
        assert call(adam(**{name: F + 2}), tensor()) == AL, name
    assert f(adam(), None, 1, None, 0) == A and f(adam(), None, -1, None, 0) == S and \
        f(adam(), None, (1 << 20) + 1, None, 0) == S
    assert f(adam(), (lm.lmhead_adamw_tensor * 1)(tensor()), 1, F + 4, 0) == AL
    e8 = dict(state_dtype=2, exp_avg_scale=F, exp_avg_sq_scale=F)
    good = tensor()
    for bad in (dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(param_dtype=2),
                dict(grad_dtype=2), dict(state_dtype=0), dict(state_dtype=3), dict(reserved=1), dict(exp_avg_scale=F),
                dict(exp_avg_sq_scale=F), dict(e8, exp_avg_scale=None), dict(e8, exp_avg_sq_scale=None)):
        assert call(adam(), good, tensor(**bad)) == A, bad
    for bad in (dict(numel=-1), dict(numel=1 << 35)):
        assert call(adam(), good, tensor(**bad)) == S, bad
    for bad in (dict(param=F + 1), dict(grad=F + 1), dict(param=F + 2, param_dtype=1), dict(grad=F + 2, grad_dtype=1),
                dict(exp_avg=F + 2), dict(exp_avg_sq=F + 2), dict(copy=F + 1), dict(e8, exp_avg_scale=F + 2),
                dict(e8, exp_avg_sq_scale=F + 2)):
        assert call(adam(), good, tensor(**bad)) == AL, bad


def test_adamw_table():
    f, size = lm.lmhead_adamw_table, lm.lmhead_adamw_table_size
    assert size(0) == 0 and size(-1) == 0 and size((1 << 20) + 1) == 0
    assert size(1) == 64 + 72 and size(16) == 64 + 16 * 72 and size(17) == 128 + 17 * 72
    e8 = dict(state_dtype=2, exp_avg_scale=FAKE, exp_avg_sq_scale=FAKE)
    tensors = (lm.lmhead_adamw_tensor * 4)(tensor(numel=2049), tensor(numel=0), tensor(numel=4097, **e8), tensor())
    buf = torch.zeros(size(4), dtype=torch.uint8)
    assert f(tensors, 4, buf, size(4)) == lm.LMHEAD_OK
    assert buf[:16].view(torch.int32).tolist() == [0, 2, 2, 4]   # chunks of 2048, or of 4096 in 8 bits
    assert f(tensors, 4, buf, size(4) - 1) == W and f(tensors, 4, None, BIG) == A and f(None, 4, buf, BIG) == A
    assert f(tensors, 4, buf.data_ptr() + 4, BIG) == AL and f(None, -1, None, 0) == S
    assert f((lm.lmhead_adamw_tensor * 1)(tensor(param=None)), 1, buf, BIG) == A
    big = (lm.lmhead_adamw_tensor * 2)(*[tensor(numel=(1 << 35) - (1 << 24))] * 2)
    assert f(big, 2, buf, BIG) == S and f(big, 1, buf, BIG) == lm.LMHEAD_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device():
    D, F = lm.LMHEAD_ERR_DEVICE, FAKE
    assert lm.lmhead_embedding_fwd(emb(), F, F, None, F, None, 0, 0) == D
    assert lm.lmhead_embedding_fwd(emb(weight_dtype=2), F, F, F, F, F, 256, 0) == D
    assert lm.lmhead_embedding_bwd(emb(accumulate=1), F, F, F, F, BIG, 0) == D
    assert lm.lmhead_policy_loss_fwd(pol(), F, F, F, F, F, F, F, None, F, F, BIG, 0) == D
    assert lm.lmhead_policy_loss_fwd(pol(sequences=0, kl_weight=0.0), F, None, None, F, None, None, F, F, F, F, BIG, 0) == D
    assert lm.lmhead_policy_loss_bwd(pol(), F, F, F, F, F, F, F, F, F, 0) == D
    assert lm.lmhead_preference_loss_fwd(pref(), F, None, None, F, F, None, F, F, BIG, 0) == D
    assert lm.lmhead_preference_loss_bwd(pref(), F, F, F, F, F, 0) == D
    one = (lm.lmhead_adamw_tensor * 1)(tensor(exp_avg=F + 4, param=F + 2))
    assert lm.lmhead_adamw_step(adam(), one, 1, None, 0) == D
    assert lm.lmhead_adamw_step(adam(), None, 0, FAKE, 0) == D


def test_helpers_refuse():
    ids, w = torch.zeros(3, dtype=torch.int32), torch.zeros(8, 64, dtype=torch.bfloat16)
    x, cu = torch.zeros(4), torch.tensor([0, 2, 4], dtype=torch.int32)
    for call in (lambda: lm.embedding(ids, w), lambda: lm.embedding_backward(w, ids, 8), lambda: lm.policy_loss(x, x),
                 lambda: lm.policy_loss_backward(x[:1], x[:1], x, x), lambda: lm.preference_loss(x, cu),
                 lambda: lm.preference_loss_backward(x[:1], x[:2], 4, cu),
                 lambda: lm.adamw_plan([x], [x], [lm.adamw_state(x)])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="parameter"):
        lm.adamw_plan([], [], [])
    with pytest.raises(ValueError, match="length"):
        lm.adamw_plan([x], [], [lm.adamw_state(x)])
    with pytest.raises(ValueError, match="dtype"):
        lm.adamw_state(x, torch.bfloat16)
    s = lm.adamw_state(torch.zeros(3, 100), torch.float8_e4m3fn)
    assert s.exp_avg.shape == (3, 100) and s.exp_avg_scale.shape == (3,) and s.exp_avg.float().abs().max() == 0


class Elsewhere(torch.Tensor):
    """Reports the GPU cuda:1; no data is ever read."""
    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


class Entered(Exception):
    pass


@pytest.mark.parametrize("name,arg,count", [
    ("embedding_forward", "ids", 2), ("embedding_backward", "dout", 3), ("policy_loss_forward", "logp", 2),
    ("policy_loss_backward", "grad", 4), ("preference_loss_forward", "logp", 2),
    ("preference_loss_backward", "grad", 4)])
def test_helpers_run_on_their_tensors_device(monkeypatch, name, arg, count):
    @contextlib.contextmanager
    def device(d):
        assert torch.device(d) == torch.device("cuda", 1)
        raise Entered
        yield
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    t = torch.zeros(4).as_subclass(Elsewhere)
    fn = getattr(lm, name)
    with pytest.raises(Entered):
        fn(t, *[1] * (count - 1))
    names = inspect.unwrap(fn).__code__.co_varnames[:count]
    assert names[0] == arg
    with pytest.raises(Entered):
        fn(**{n: t if n == arg else 1 for n in names})


# ------------------------------------------------ the plain definitions

def packed(rng, n, sequences, off=0.3):
    cu = np.sort(rng.integers(0, n + 1, sequences + 1))
    targets = np.where(rng.random(n) < off, -1, 5)
    return cu, targets


@pytest.mark.parametrize("kw", [dict(), dict(reduction="sum", kl_kind="k1"), dict(reduction="sequence_mean", kl_kind="k2"),
                                dict(dual_clip=1.3, num_valid=50)])
def test_reference_policy_gradient_against_differences(kw):
    rng = np.random.default_rng(1)
    n = 60
    cu, targets = packed(rng, n, 5)
    logp, old, ref_, adv = -rng.random(n), -rng.random(n), -rng.random(n), rng.standard_normal(n)
    kw = dict(kw, kl_weight=0.3)
    args = (adv, old, ref_, targets, cu)
    _, _, dlogp, _ = ref.policy(logp, *args, **kw)
    assert np.count_nonzero(dlogp) > 5
    h = 1e-6
    for t in range(n):
        up, down = logp.copy(), logp.copy()
        up[t] += h
        down[t] -= h
        d = (ref.policy(up, *args, **kw)[0] - ref.policy(down, *args, **kw)[0]) / (2 * h)
        assert abs(d - dlogp[t]) < 1e-7, t


@pytest.mark.parametrize("kw", [dict(label_smoothing=0.1), dict(kind="hinge", beta=0.2, margin=0.3),
                                dict(kind="squared", average=True), dict(average=True, margin=0.5, num_pairs=7)])
def test_reference_preference_gradient_against_differences(kw):
    rng = np.random.default_rng(2)
    n = 80
    cu, targets = packed(rng, n, 8)
    logp, ref_ = -rng.random(n), -rng.random(n)
    _, rewards, dlogp = ref.preference(logp, cu, ref_, targets, **kw)
    assert np.count_nonzero(dlogp) > 5
    h = 1e-6
    for t in range(n):
        up, down = logp.copy(), logp.copy()
        up[t] += h
        down[t] -= h
        d = (ref.preference(up, cu, ref_, targets, **kw)[0] - ref.preference(down, cu, ref_, targets, **kw)[0]) / (2 * h)
        # a second difference of the squared loss: h^2 times its third derivative is nil, rounding ~ 1e-16 loss / h
        assert abs(d - dlogp[t]) < 1e-7, t


def test_reference_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(3)
    ids, w = rng.integers(-2, 7, 30), rng.standard_normal((7, 5))
    dout = rng.standard_normal((30, 5))
    s, a, c = ref.embedding_grad(ids, dout, 7, 1.5)
    assert abs((ref.embedding(ids, w, 1.5) * dout).sum() - (s * w).sum()) < 1e-12
    assert c.sum() == (ids >= 0).sum() and (a >= abs(s)).all()


def test_reference_adamw_first_step():
    p, m, v, _ = ref.adamw(np.array([1.0]), np.array([0.3]), 0.0, 0.0, 1, 0.01, 0.9, 0.999, 1e-12, 0.5)
    # the first step's quotient is the gradient's sign
    assert abs(p[0] - (1.0 - 0.01 * 0.5 - 0.01)) < 1e-10 and abs(m[0] - 0.03) < 1e-15 and abs(v[0] - 9e-5) < 1e-15
