"""Refusals and sizes of include/lmhead_decode.h, on the host: every call here
fails validation (fake addresses are never dereferenced) or, with valid
arguments and no device, ends in LMHEAD_ERR_DEVICE. Also the plain definitions
the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import decode_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
BIG = 1 << 40
A, S, AL, W = lm.LMHEAD_ERR_ARG, lm.LMHEAD_ERR_SHAPE, lm.LMHEAD_ERR_ALIGN, lm.LMHEAD_ERR_WORKSPACE


def test_library_exports_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "lmhead_decode.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(lmhead_[a-z_0-9]+)\s*\(", text)))
    assert names == ["lmhead_logits_fp8", "lmhead_logits_fp8_workspace_size", "lmhead_quantize_fp8",
                     "lmhead_rms_norm_bwd", "lmhead_rms_norm_bwd_workspace_size", "lmhead_rms_norm_fwd",
                     "lmhead_sample", "lmhead_sample_workspace_size"]
    L = ctypes.CDLL(lm.LIB_PATH)
    for name in names:
        assert hasattr(L, name) and hasattr(lm, name), name


def norm(**kw):
    d = dict(n=4, hidden=256, eps=1e-6, weight_offset=0.0, weight_dtype=0, reserved=0)
    d.update(kw)
    return lm.lmhead_norm(*d.values())


def test_norm_refusals():
    f, F = lm.lmhead_rms_norm_fwd, FAKE
    ok = dict(x=F, residual=F, weight=F, residual_out=F, y=F + 4096, q=F, scale=F, rstd=F, stream=0)

    def call(p, **kw):
        return f(p, *{**ok, **kw}.values())
    for bad in (dict(reserved=1), dict(weight_dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(weight_offset=float("inf")), dict(weight_offset=float("nan"))):
        assert call(norm(**bad)) == A, bad
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(hidden=0), dict(hidden=100), dict(hidden=65600)):
        assert call(norm(**bad)) == S, bad
    assert call(norm(hidden=192)) == S                      # 8-bit output: whole blocks
    assert call(norm(), q=None) == A and call(norm(), scale=None) == A
    assert call(norm(), residual=None) == A                 # residual_out without residual
    assert call(norm(), y=F) == A                           # y and residual_out in one buffer
    assert call(norm(), x=None) == A and call(norm(), weight=None) == A
    assert call(norm(), residual_out=None, y=None, q=None, scale=None, rstd=None) == A
    for name in ("x", "residual", "weight", "residual_out", "y", "q", "scale", "rstd"):
        assert call(norm(), **{name: F + (2 if name in ("scale", "rstd") else 8) + (4096 if name == "y" else 0)}) == AL, name


def test_norm_backward_refusals():
    f, F = lm.lmhead_rms_norm_bwd, FAKE
    ok = dict(dy=F, r=F, weight=F, rstd=F, dres=F, dx=F, dw=F, ws=F, bytes=BIG, stream=0)

    def call(p, **kw):
        return f(p, *{**ok, **kw}.values())
    size = lm.lmhead_rms_norm_bwd_workspace_size
    assert size(norm(hidden=100)) == 0 and size(norm(n=0)) > 0
    assert size(norm(n=1 << 20)) == size(norm(n=512)) == 4 * 512 * 256
    for name in ("dy", "r", "weight", "rstd"):
        assert call(norm(), **{name: None}) == A, name
    assert call(norm(), ws=None) == A
    assert call(norm(), bytes=size(norm()) - 1) == W
    for name in ("dy", "r", "weight", "rstd", "dres", "dx", "dw"):
        assert call(norm(), **{name: F + 2}) == AL, name
    assert call(norm(), ws=F + 128) == AL


def test_quantize_refusals():
    f, F = lm.lmhead_quantize_fp8, FAKE
    assert f(4, 256, 64, F, F, F, 0) == A
    for rows, cols in ((-1, 256), ((1 << 30) + 1, 256), (4, 0), (4, 192), (4, 65664)):
        assert f(rows, cols, 1, F, F, F, 0) == S, (rows, cols)
    # one workgroup per 128 x 128 block: at most 2^24 - 1 of them
    assert f(128 * ((1 << 24) // 512 + 1), 65536, 128, F, F, F, 0) == S
    assert f(4, 256, 1, None, F, F, 0) == A and f(4, 256, 1, F, None, F, 0) == A and f(4, 256, 1, F, F, None, 0) == A
    assert f(4, 256, 1, F + 2, F, F, 0) == AL and f(4, 256, 1, F, F, F + 2, 0) == AL


def fp8(**kw):
    d = dict(n=4, vocab=1000, hidden=256, ld=1000, out_dtype=1, reserved=0)
    d.update(kw)
    return lm.lmhead_fp8_problem(*d.values())


def test_logits_refusals():
    f, F, size = lm.lmhead_logits_fp8, FAKE, lm.lmhead_logits_fp8_workspace_size
    for bad in (dict(reserved=1), dict(out_dtype=2)):
        assert f(fp8(**bad), F, F, F, F, F, F, BIG, 0) == A and size(fp8(**bad)) == 0
    for bad in (dict(n=-1), dict(n=(1 << 24) + 1), dict(vocab=0), dict(ld=999), dict(hidden=64), dict(hidden=192),
                dict(hidden=65664), dict(n=1 << 20, vocab=1 << 20, ld=1 << 20), dict(ld=(1 << 32) + 1)):
        assert f(fp8(**bad), F, F, F, F, F, F, BIG, 0) == S and size(fp8(**bad)) == 0, bad
    for i in range(6):
        assert f(fp8(), *[None if j == i else F for j in range(6)], BIG, 0) == A
        assert f(fp8(), *[F + (2 if i in (1, 3, 4) else 8) if j == i else F for j in range(6)], BIG, 0) == AL
    assert f(fp8(), F, F, F, F, F, F, 0, 0) == W


def samp(**kw):
    d = dict(n=4, vocab=1000, ld=1000, logits_dtype=1, top_k=0, temperature=0.0, top_p=0.0, min_p=0.0, reserved=0,
             rt=None, rk=None, rp=None, rm=None)
    d.update(kw)
    return lm.lmhead_sample_problem(*d.values())


def test_sample_refusals():
    f, F, size = lm.lmhead_sample, FAKE, lm.lmhead_sample_workspace_size
    nan = float("nan")
    for bad in (dict(reserved=1), dict(logits_dtype=2), dict(temperature=-1.0), dict(temperature=nan),
                dict(temperature=float("inf")), dict(top_p=1.5), dict(top_p=-0.1), dict(top_p=nan), dict(min_p=1.1),
                dict(min_p=nan), dict(top_k=-1)):
        assert f(samp(**bad), F, F, F, F, F, BIG, 0) == A and size(samp(**bad)) == 0, bad
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(ld=10)):
        assert f(samp(**bad), F, F, F, F, F, BIG, 0) == S and size(samp(**bad)) == 0, bad
    for i in (0, 1, 2, 4):   # logprob (3) may be NULL
        assert f(samp(), *[None if j == i else F for j in range(5)], BIG, 0) == A
    assert f(samp(), F + 2, F, F, F, F, BIG, 0) == AL and f(samp(logits_dtype=0), F + 1, F, F, F, F, BIG, 0) == AL
    assert f(samp(), F, F, F, F, F + 16, BIG, 0) == AL
    for name in ("rt", "rk", "rp", "rm"):
        assert f(samp(**{name: F + 2}), F, F, F, F, F, BIG, 0) == AL, name
    assert f(samp(), F, F, F, F, F, 0, 0) == W


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_no_device():
    D, F = lm.LMHEAD_ERR_DEVICE, FAKE
    assert lm.lmhead_rms_norm_fwd(norm(), F, None, F, None, F, None, None, None, 0) == D
    assert lm.lmhead_rms_norm_bwd(norm(), F, F, F, F, None, F, None, None, 0, 0) == D
    assert lm.lmhead_quantize_fp8(4, 256, 1, F, F, F, 0) == D
    assert lm.lmhead_logits_fp8(fp8(), F, F, F, F, F, F, BIG, 0) == D
    assert lm.lmhead_sample(samp(), F, F, F, F, F, BIG, 0) == D


def test_helpers_refuse_cpu_tensors():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    w = torch.ones(256, dtype=torch.bfloat16)
    q = torch.zeros(2, 256, dtype=torch.float8_e4m3fn)
    s = torch.ones(2, 2)
    for call in (lambda: lm.rms_norm(x, w), lambda: lm.rms_norm_quant(x, w), lambda: lm.quantize_fp8(x),
                 lambda: lm.logits_fp8(q, s, q, s), lambda: lm.sample(torch.zeros(2, 8), torch.zeros(2)),
                 lambda: lm.rms_norm_backward(x, x, w, torch.ones(2))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_reference_sampler_small_cases():
    x = np.log(np.array([0.1, 0.4, 0.4, 0.1]))
    # index order: running sums 0.1, 0.5, 0.9, 1.0
    assert [ref.sample_row(x, u)[0] for u in (0.0, 0.099, 0.101, 0.499, 0.501, 0.899, 0.901, 0.999)] == \
        [0, 0, 1, 1, 2, 2, 3, 3]
    assert ref.sample_row(x, 0.99, top_k=1)[0] == 1          # equal logits: the lowest index first
    assert ref.sample_row(x, 0.99, top_k=3)[0] == 2 and ref.sample_row(x, 0.01, top_k=3)[0] == 0
    assert ref.sample_row(x, 0.999, top_p=0.3)[0] == 1       # 0.4 already reaches 0.3
    assert ref.sample_row(x, 0.999, top_p=0.5)[0] == 2
    assert ref.sample_row(x, 0.999, min_p=0.5)[0] == 2 and ref.sample_row(x, 0.0, min_p=0.5)[0] == 1
    assert ref.sample_row(np.full(4, -np.inf), 0.5) == (-1, 0.0)
    assert abs(ref.sample_row(x, 0.2, tau=0.5)[1] - np.log(0.16 / 0.34)) < 1e-12


def test_reference_norm_gradients_against_differences():
    rng = np.random.default_rng(3)
    x, w, dy = rng.standard_normal((3, 64)), 1 + 0.1 * rng.standard_normal(64), rng.standard_normal((3, 64))

    def loss(x, w):
        return (ref.norm(x, None, w, 1e-3, 0.5)[2] * dy).sum()
    r, rstd, _ = ref.norm(x, None, w, 1e-3, 0.5)
    dx, dw = ref.norm_backward(dy, r, w, rstd, None, 0.5)
    h = 1e-5
    for _ in range(5):
        vx, vw = rng.standard_normal(x.shape), rng.standard_normal(64)
        d = (loss(x + h * vx, w + h * vw) - loss(x - h * vx, w - h * vw)) / (2 * h)
        assert abs(d - ((dx * vx).sum() + (dw * vw).sum())) < 1e-7 * max(1.0, abs(d))


def test_a_bad_problem_is_named_by_its_entry():
    """Where the size function says 0, the helpers raise the entry's own status."""
    from chunked_lm_head_amd import decode
    for entry, p, pointers, want in ((lm.lmhead_sample, samp(top_p=1.5), 5, A), (lm.lmhead_sample, samp(vocab=0), 5, S),
                                     (lm.lmhead_sample, samp(n=0, top_k=-2), 5, A), (lm.lmhead_logits_fp8, fp8(hidden=192), 6, S),
                                     (lm.lmhead_rms_norm_bwd, norm(eps=-1.0), 8, A), (lm.lmhead_rms_norm_bwd, norm(hidden=100), 8, S)):
        with pytest.raises(lm.LMHeadError) as e:
            decode._workspace(None, 0, "cpu", entry, p, pointers)
        assert e.value.status == want and entry.__name__ in str(e.value)
