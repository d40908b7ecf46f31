"""RMS norm (forward, 8-bit output, backward) and the block quantiser against
their 64-bit definitions.

Tolerances. A bf16 result is off by at most half a step, 2^-8 of its value; an
e4m3 value by 2^-4 of it, or half of the smallest step, 2^-10, times the scale.
fp32 intermediates: a sum of h squares in fp32 is off by at most (h / 256 + 24)
2^-24 of itself on this reduction (at most h / lanes + a tree of ~24 additions;
at most 128 per lane), i.e. under 1e-5; rstd by half of it; products by a few
2^-24. FP = 2e-5 covers them."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import decode_ref as ref

pytestmark = pytest.mark.gpu
FP = 2e-5
BF = 2.0 ** -8 * 1.01


def bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(n, hidden, seed, residual=True, weight=torch.bfloat16, offset=0.0):
    rng = np.random.default_rng(seed)
    x = bf(rng.standard_normal((n, hidden)))
    res = bf(3.0 * rng.standard_normal((n, hidden))) if residual else None
    w = torch.from_numpy((1.0 - offset + 0.1 * rng.standard_normal(hidden)).astype(np.float32)).to(weight).cuda()
    return x, res, w, rng


def check_quantised(q, s, y, block_rows):
    want = ref.block_scales(y, block_rows)
    got = f64(s)
    assert got.shape == want.shape
    assert (np.abs(got - want) <= FP * want).all()
    each = ref.spread_scales(got, block_rows, y.shape[0])
    v = f64(q) * each
    assert (np.abs(v - y) <= np.abs(y) * (2.0 ** -4 + FP) + each * 2.0 ** -10 * 1.01).all()


SHAPES = [(1, 128), (5, 512), (3, 640), (9, 1024), (2, 1152), (33, 2048), (4, 2176), (1, 4096), (70, 4096), (3, 8192),
          (2, 8320), (2, 16384), (3, 24576), (1, 65536)]


@pytest.mark.parametrize("n,hidden", SHAPES)
@pytest.mark.parametrize("residual,weight,offset", [(True, torch.bfloat16, 0.0), (False, torch.float32, 1.0)])
def test_forward(n, hidden, residual, weight, offset):
    x, res, w, _ = inputs(n, hidden, n + hidden, residual, weight, offset)
    f = lm.rms_norm_forward(x, w, res, eps=1e-5, weight_offset=offset, out_fp8=True)
    r, rstd, y = ref.norm(f64(x), None if res is None else f64(res), f64(w), 1e-5, offset)
    if residual:
        assert np.array_equal(f64(f.residual_out), r)
    else:
        assert f.residual_out is None
    assert (np.abs(f64(f.rstd) - rstd) <= FP * rstd).all()
    assert (np.abs(f64(f.y) - y) <= (BF + FP) * np.abs(y)).all()
    check_quantised(f.q, f.scale, y, 1)
    again = lm.rms_norm_forward(x, w, res, eps=1e-5, weight_offset=offset, out_fp8=True)
    for a, b in zip(f, again):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q, s, r2 = lm.rms_norm_quant(x, w, res, eps=1e-5, weight_offset=offset)
    assert torch.equal(q.view(torch.uint8), f.q.view(torch.uint8)) and torch.equal(s, f.scale)


def test_hidden_that_is_no_whole_block():
    x, res, w, _ = inputs(6, 192, 1)
    f = lm.rms_norm_forward(x, w, res)
    _, _, y = ref.norm(f64(x), f64(res), f64(w), 1e-6, 0.0)
    assert (np.abs(f64(f.y) - y) <= (BF + FP) * np.abs(y)).all()
    with pytest.raises(lm.LMHeadError):
        lm.rms_norm_quant(x, w, res)


def test_zero_rows_zero_blocks_and_bad_values():
    x, _, w, _ = inputs(5, 256, 2, False)
    x[0] = 0
    x[1, :128] = 0
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    f = lm.rms_norm_forward(x, w, eps=1e-6, out_fp8=True)
    assert (f.y[0] == 0).all() and (f.q[0].float() == 0).all() and (f.scale[0] == 1).all()
    assert f.scale[1, 0] == 1 and (f.q[1, :128].float() == 0).all() and (f.q[1, 128:].float() != 0).any()
    # a bad value shows in its own row and in no other
    assert f.y[2].isnan().all() and f.q[2].float().isnan().all()
    assert f.y[3, 5].isnan() and f.q[3, 5].float().isnan()
    _, _, y = ref.norm(f64(x[4:]), None, f64(w), 1e-6, 0.0)
    assert (np.abs(f64(f.y[4:]) - y) <= (BF + FP) * np.abs(y)).all()


def test_in_place_residual_stream():
    x, res, w, _ = inputs(37, 2048, 4)
    want = lm.rms_norm_forward(x, w, res)
    p = lm.lmhead_norm(37, 2048, 1e-6, 0.0, lm.DTYPE_BF16, 0)
    for stream_in_x in (True, False):
        a, b = x.clone(), res.clone()
        y = torch.empty_like(x)
        out = a if stream_in_x else b
        assert lm.lmhead_rms_norm_fwd(p, a, b, w, out, y, None, None, None) == lm.LMHEAD_OK
        assert torch.equal(out, want.residual_out) and torch.equal(y, want.y)
    a = x.clone()
    assert lm.lmhead_rms_norm_fwd(p, a, None, w, None, a, None, None, None) == lm.LMHEAD_OK
    assert torch.equal(a, lm.rms_norm_forward(x, w).y)


@pytest.mark.parametrize("n,hidden", [(1, 64), (3, 192), (5, 512), (2050, 512), (9, 1024), (700, 2048), (4, 2176),
                                      (1100, 4096), (3, 8192), (5, 16384), (3, 24576), (2, 65536)])
@pytest.mark.parametrize("residual,weight,offset", [(True, torch.bfloat16, 0.0), (False, torch.float32, 1.0)])
def test_backward(n, hidden, residual, weight, offset):
    x, res, w, rng = inputs(n, hidden, 7 * n + hidden, residual, weight, offset)
    dy, dr = bf(rng.standard_normal((n, hidden))), bf(rng.standard_normal((n, hidden))) if residual else None
    f = lm.rms_norm_forward(x, w, res, eps=1e-5, weight_offset=offset)
    r = f.residual_out if residual else x
    dx, dw = lm.rms_norm_backward(dy, r, w, f.rstd, dr, offset)
    rf, rstd, _ = ref.norm(f64(r), None, f64(w), 1e-5, offset)
    wx, ww = ref.norm_backward(f64(dy), rf, f64(w), rstd, None if dr is None else f64(dr), offset)
    g = np.abs(f64(dy) * (offset + f64(w)))
    h = np.abs(rf * rstd[:, None])
    # dx = rstd (g - h mean(g h)) + dr: each term to FP of its own size
    size = rstd[:, None] * (g + h * (g * h).mean(1, keepdims=True)) + (0 if dr is None else np.abs(f64(dr)))
    assert (np.abs(f64(dx) - wx) <= BF * np.abs(wx) + FP * size).all()
    # fp32 sums over n rows: n / 512 per group, then 32, 16
    tol = (n / 512 + 60) * 2.0 ** -24 * (np.abs(f64(dy)) * h).sum(0) + FP * (np.abs(f64(dy)) * h).sum(0)
    if weight == torch.bfloat16:
        tol = tol + BF * np.abs(ww)
    assert dw.dtype == weight and (np.abs(f64(dw) - ww) <= tol).all()
    dx2, dw2 = lm.rms_norm_backward(dy, r, w, f.rstd, dr, offset)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    # either side alone
    assert torch.equal(lm.rms_norm_backward(dy, r, w, f.rstd, dr, offset, need_dweight=False)[0], dx)
    assert torch.equal(lm.rms_norm_backward(dy, r, w, f.rstd, dr, offset, need_dx=False)[1], dw)
    # dx over dy's buffer
    p = lm.lmhead_norm(n, hidden, 0.0, offset, lm.DTYPE_F32 if weight == torch.float32 else lm.DTYPE_BF16, 0)
    buf = dy.clone()
    assert lm.lmhead_rms_norm_bwd(p, buf, r, w, f.rstd, dr, buf, None, None, 0) == lm.LMHEAD_OK
    assert torch.equal(buf, dx)


def test_gradient_against_differences():
    """sum(dy y) along random directions, differences of the 64-bit forward: dx
    is bf16, so the product with v is off by at most 2^-8 sum |dx v| plus the
    fp32 part; the difference quotient by O(h^2) ~ 1e-8."""
    n, hidden = 4, 256
    x, _, w, rng = inputs(n, hidden, 11, False, torch.float32)
    dy = bf(rng.standard_normal((n, hidden)))
    f = lm.rms_norm_forward(x, w, eps=1e-3)
    dx, dw = lm.rms_norm_backward(dy, x, w, f.rstd)
    X, W, D = f64(x), f64(w), f64(dy)
    for _ in range(4):
        vx, vw = rng.standard_normal(X.shape), rng.standard_normal(W.shape)
        h = 1e-4
        d = ((ref.norm(X + h * vx, None, W + h * vw, 1e-3, 0.0)[2]
              - ref.norm(X - h * vx, None, W - h * vw, 1e-3, 0.0)[2]) * D).sum() / (2 * h)
        got = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
        tol = BF * np.abs(f64(dx) * vx).sum() + FP * (np.abs(D).sum() + np.abs(f64(dw) * vw).sum()) + 1e-6
        assert abs(d - got) <= tol


def test_autograd_norm_in_front_of_the_loss():
    """rms_norm -> ce_loss: the gradients reach x, the residual and the weight as
    the explicit calls give them, also through the residual stream's other use."""
    n, hidden, vocab = 40, 256, 1000
    x, res, w, rng = inputs(n, hidden, 13)
    W = bf(0.05 * rng.standard_normal((vocab, hidden)))
    t = torch.from_numpy(rng.integers(0, vocab, n).astype(np.int32)).cuda()
    other = bf(rng.standard_normal((n, hidden)))
    for leaf in (x, res, w):
        leaf.requires_grad_(True)
    y, r = lm.rms_norm(x, w, res)
    loss = lm.ce_loss(y, W, t, chunk=256) + (r.float() * other.float()).sum()
    loss.backward()
    with torch.no_grad():
        f = lm.rms_norm_forward(x, w, res)
        _, lse, _ = lm.ce_loss_forward(f.y, W, t, 256)
        one = torch.ones(1, device="cuda")
        dy, _ = lm.backward(lm.ENTRY_CE_MEAN, f.y, W, t, lse, one, 256, need_dW=False)
        dx, dw = lm.rms_norm_backward(dy, f.residual_out, w, f.rstd, other)
    assert torch.equal(x.grad, dx) and torch.equal(res.grad, dx) and torch.equal(w.grad, dw)
    # without a residual, x alone needing a gradient
    x2 = x.detach().clone().requires_grad_(True)
    lm.rms_norm(x2, w.detach()).float().sum().backward()
    assert x2.grad is not None and torch.isfinite(x2.grad).all()
    # only the residual stream used
    x3, r3 = x.detach().clone().requires_grad_(True), res.detach().clone().requires_grad_(True)
    lm.rms_norm(x3, w.detach(), r3)[1].float().sum().backward()
    assert torch.equal(x3.grad, torch.ones_like(x3)) and torch.equal(r3.grad, torch.ones_like(r3))


def test_one_tensor_in_two_places():
    """x as its own residual, and gradients that do not share memory."""
    x, dy = (torch.randn(9, 256, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(256, device="cuda").to(torch.bfloat16)
    f = lm.rms_norm_forward(x, w, x)
    dx, _ = lm.rms_norm_backward(dy, f.residual_out, w, f.rstd)
    a = x.clone().requires_grad_()
    y, _ = lm.rms_norm(a, w, a)
    y.backward(dy)
    assert torch.equal(y, f.y) and torch.equal(a.grad, dx + dx)
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    lm.rms_norm(a, w, b)[0].backward(dy)
    assert torch.equal(a.grad, dx) and torch.equal(b.grad, dx)
    a.grad.zero_()
    assert torch.equal(b.grad, dx)
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    lm.rms_norm(a, w, b)[1].backward(dy)       # the residual stream alone
    assert torch.equal(a.grad, dy) and torch.equal(b.grad, dy)


def test_empty():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q, s, r = lm.rms_norm_quant(x, w, x)
    assert q.shape == (0, 256) and s.shape == (0, 2) and r.shape == (0, 256)
    dx, dw = lm.rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 256) and (dw == 0).all()
    q, s = lm.quantize_fp8(x, 128)
    assert q.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.parametrize("rows,cols,block_rows", [(1, 128, 1), (7, 384, 1), (300, 2048, 1), (1, 128, 128), (127, 256, 128),
                                                  (128, 256, 128), (129, 1152, 128), (1000, 640, 128)])
def test_quantize(rows, cols, block_rows):
    rng = np.random.default_rng(rows + cols)
    x = bf(rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-20, 20, (rows, 1))))
    x[0, :128] = 0
    if rows > 2:
        x[2] *= 1e-38          # blocks near the smallest normal number
    q, s = lm.quantize_fp8(x, block_rows)
    check_quantised(q, s, f64(x), block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_bad_values(block_rows):
    x = torch.ones(256, 256, dtype=torch.bfloat16, device="cuda")
    x[3, 7] = float("nan")
    x[200, 130] = float("inf")
    q, s = lm.quantize_fp8(x, block_rows)
    v = q.float() * (s.repeat_interleave(128, 1) if block_rows == 1
                     else s.repeat_interleave(128, 0).repeat_interleave(128, 1))
    assert v[3, 7].isnan() and not torch.isfinite(v[200, 130])
    clean = torch.ones(256, 256, dtype=torch.bool, device="cuda")
    if block_rows == 1:
        clean[3, :128] = clean[200, 128:] = False
    else:
        clean[:128, :128] = clean[128:, 128:] = False
    assert (v[clean] == 1.0).all()


def e4m3_of(v):
    """Nearest e4m3 value (ties to even) of fp64 numbers within +-448."""
    mag = np.abs(v)
    e = np.maximum(np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6.0)
    step = np.exp2(e - 3.0)
    return np.sign(v) * np.minimum(np.round(mag / step) * step, 448.0)


def quotients(top):
    """Blocks of 128 fp32 values, the first of each the largest: every bf16
    mantissa below it, at eight binary orders and both signs. Their number, and
    the quotients and scales as one fp32 division each."""
    m = (128 + np.arange(128)) / 128.0
    orders = np.exp2(-np.arange(1, 9))[:, None] * m * np.where(np.arange(128) % 3 == 0, -1.0, 1.0)
    low, high = orders[:, :64], orders[:, 64:]
    blocks = np.zeros((16, 128))
    blocks[:8, 1:65], blocks[8:, 1:65] = low, high
    blocks[:, 65:] = -blocks[:, 2:65]
    x = blocks[None] * np.exp2(np.floor(np.log2(top)))[:, None, None]
    x[:, :, 0] = top[:, None]
    x = x.astype(np.float32)
    s = (np.abs(x).max(2) / np.float32(448)).astype(np.float32)
    return x.reshape(len(top), -1), s, (x / s[:, :, None]).astype(np.float64).reshape(len(top), -1)


@pytest.mark.parametrize("order", [0, 7, -60, 90, -110, 127])
def test_quotients_are_one_division(order):
    """q is the e4m3 rounding of the fp32 quotient y / s, s that of max / 448: a
    product with 1 / s is off by a step where the quotient is a tie (153 of 204
    is 336, halfway between 320 and 352)."""
    top = (128 + np.arange(128)) / 128.0 * 2.0 ** order
    x, s, want = quotients(top)
    want = e4m3_of(want)
    q, scale = lm.quantize_fp8(bf(x), 1)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(f64(q), want), np.argwhere(f64(q) != want)[:5]
    # the same rows as 128 x 128 blocks of one row each
    q, scale = lm.quantize_fp8(bf(x).repeat_interleave(128, 0), 128)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(f64(q), np.repeat(want, 128, 0))
    # a row of ones has rstd 1 at eps 0, so the norm's y is the weight
    for i in (0, 10, 63, 76, 80, 127):
        w = torch.from_numpy(x[i]).cuda()
        q, scale, _ = lm.rms_norm_quant(torch.ones(1, x.shape[1], dtype=torch.bfloat16, device="cuda"), w, eps=0.0)
        assert np.array_equal(scale.cpu().numpy()[0], s[i]) and np.array_equal(f64(q)[0], want[i]), i


def test_refusals_keep_the_entry_status():
    x, _, w, _ = inputs(3, 256, 1, False)
    rstd = torch.ones(3, device="cuda")
    with pytest.raises(lm.LMHeadError) as e:
        lm.rms_norm_backward(x, x, w, rstd, weight_offset=float("inf"))
    assert e.value.status == lm.LMHEAD_ERR_ARG
    y = torch.zeros(3, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lm.LMHeadError) as e:
        lm.rms_norm_backward(y, y, w[:96], rstd)
    assert e.value.status == lm.LMHEAD_ERR_SHAPE
