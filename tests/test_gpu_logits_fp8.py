"""Logits from 8-bit operands against the 64-bit product of the values they
stand for.

Tolerance. Products of e4m3 values are exact in fp32; a block's 128 products
and the blocks' sums are fp32 additions, each off by at most one step (2^-23,
truncation allowed) of a partial sum that the sum of magnitudes bounds: (128 +
blocks) 2^-23 sum |a w|. A bf16 output adds half a step, 2^-8; with more than 64
rows it may come from the 8-bit matrix instructions, which cut the eight products
of aligned consecutive columns off 13 bits below the power of two of the
largest one: at most 8 * 2^-13 of each eight's largest |a w| more
(test_the_cut_off measures that the instructions do no worse)."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import decode_ref as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def operand(rows, cols, block_rows, rng):
    q = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32) * 100).clamp(-448, 448)
    q = q.to(torch.float8_e4m3fn).cuda()
    s = torch.from_numpy(np.exp(rng.uniform(-3, 3, (-(-rows // block_rows), cols // 128))).astype(np.float32)).cuda()
    return q, s


def check(out, a, sa, w, sw):
    A = f64(a) * ref.spread_scales(f64(sa), 1, a.shape[0])
    B = f64(w) * ref.spread_scales(f64(sw), 128, w.shape[0])
    z, size = A @ B.T, np.abs(A) @ np.abs(B).T
    tol = (128 + a.shape[1] // 128) * 2.0 ** -23 * size
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * 1.01 * np.abs(z)
        if a.shape[0] > 64:
            for k in range(0, a.shape[1], 8):
                tol += 8 * 2.0 ** -13 * np.max(np.abs(A[:, None, k:k + 8] * B[None, :, k:k + 8]), axis=2)
    bad = ~(np.abs(f64(out) - z) <= tol)   # NaN is bad too
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], np.abs(f64(out) - z).max())


SHAPES = [(1, 1, 128), (1, 1000, 256), (3, 130, 384), (5, 16, 128), (15, 257, 512), (16, 128, 640), (17, 1000, 256),
          (32, 63, 1152), (33, 2050, 128), (64, 512, 4096), (65, 300, 256), (80, 260, 1280), (100, 129, 1280), (128, 1000, 512),
          (200, 700, 256), (257, 513, 384), (300, 1100, 2048), (513, 260, 128), (300, 9000, 128), (1030, 1030, 256)]


@pytest.mark.parametrize("n,vocab,hidden", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_definition(n, vocab, hidden, dtype):
    print(f"[logits] n={n} vocab={vocab} hidden={hidden} {dtype}", flush=True)
    rng = np.random.default_rng(n * 7 + vocab + hidden)
    a, sa = operand(n, hidden, 1, rng)
    w, sw = operand(vocab, hidden, 128, rng)
    out = lm.logits_fp8(a, sa, w, sw, out_dtype=dtype)
    check(out, a, sa, w, sw)
    assert torch.equal(out, lm.logits_fp8(a, sa, w, sw, out_dtype=dtype))


# columns enough for the tiles on both output types (few columns go through the stream in sets of 64 rows)
# (fp32 output: from n = 130 on; the smaller n go through the stream too, see LONG for their tiles)
TILED = [(65, 16400, 256), (70, 16500, 128), (100, 16700, 384), (128, 16385, 640), (130, 22001, 128), (200, 16500, 256),
         (257, 13300, 128), (300, 13200, 384), (513, 7300, 128), (1030, 4100, 256), (2048, 2200, 128)]


@pytest.mark.parametrize("n,vocab,hidden", TILED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tiles_against_definition(n, vocab, hidden, dtype):
    test_against_definition(n, vocab, hidden, dtype)


@pytest.mark.parametrize("n,vocab,hidden", [(65, 17, 128), (129, 2000, 256), (700, 1000, 384), (1000, 33, 1280),
                                            (2048, 1024, 128), (16384, 20, 128), (16400, 20, 128), (64, 300, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sets_of_rows_against_definition(n, vocab, hidden, dtype):
    test_against_definition(n, vocab, hidden, dtype)


@pytest.mark.parametrize("n", [70, 200, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ld", [16500, 16501, 16504, 16512])
@pytest.mark.parametrize("first", [0, 1, 4])
def test_tiles_in_slices(n, dtype, ld, first):
    """Row strides and first columns of every alignment: the values of whole rows, and the rest stays."""
    rng = np.random.default_rng(9)
    vocab = 16490
    a, sa = operand(n + 1, 128, 1, rng)
    w, sw = operand(vocab, 128, 128, rng)
    buf = torch.full((n + 1, ld), 7.0, dtype=dtype, device="cuda")
    out = lm.logits_fp8(a[1:], sa[1:], w, sw, out=buf[:n, first:first + vocab])
    assert torch.equal(out, lm.logits_fp8(a[1:], sa[1:], w, sw, out_dtype=dtype))
    assert (buf[:n, :first] == 7.0).all() and (buf[:n, first + vocab:] == 7.0).all() and (buf[n] == 7.0).all()


@pytest.mark.parametrize("vocab", [16, 9008])
def test_the_cut_off(vocab):
    """2^16 beside seven 2^e in one eight of columns, -2^16 beside seven 2^e in
    the next, 2^e alone in the other 14: the large ones cancel, so the sum shows
    how much of the small ones arrived. From 2^(16 - 13) up all of them do;
    smaller ones may be lost beside 2^16, and only there."""
    n = 80
    for e, whole in ((4, True), (3, True), (2, False), (-6, False)):
        a, w = torch.zeros(n, 128), torch.zeros(vocab, 128)
        a[:, :], w[:, :] = 2.0 ** (e // 2), 2.0 ** (e - e // 2)
        a[:, 0], w[:, 0] = 256.0, 256.0
        a[:, 8], w[:, 8] = 256.0, -256.0
        out = lm.logits_fp8(a.to(torch.float8_e4m3fn).cuda(), torch.ones(n, 1, device="cuda"),
                            w.to(torch.float8_e4m3fn).cuda(), torch.ones(-(-vocab // 128), 1, device="cuda"))
        got = f64(out) / 2.0 ** e
        least = 126 if whole else 112
        assert (got >= least * (1 - 2.0 ** -8)).all() and (got <= 126 * (1 + 2.0 ** -8)).all(), (e, got[0, 0])


@pytest.mark.parametrize("n", [2, 40, 150, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ld", [333, 335, 512])
def test_row_stride_leaves_the_rest(n, dtype, ld):
    rng = np.random.default_rng(5)
    a, sa = operand(n, 256, 1, rng)
    w, sw = operand(333, 256, 128, rng)
    buf = torch.full((n + 1, ld), 7.0, dtype=dtype, device="cuda")
    out = lm.logits_fp8(a, sa, w, sw, out=buf[:n, :333])
    check(out, a, sa, w, sw)
    assert (buf[:n, 333:] == 7.0).all() and (buf[n] == 7.0).all()


@pytest.mark.parametrize("n", [3, 40, 70, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_slices_of_rows_and_columns(n, dtype):
    """Rows and their scales from the second on, and an output that starts at the
    second column: aligned to their elements only."""
    rng = np.random.default_rng(8)
    a, sa = operand(n + 1, 128, 1, rng)
    w, sw = operand(300, 128, 128, rng)
    buf = torch.full((n, 304), 7.0, dtype=dtype, device="cuda")
    out = lm.logits_fp8(a[1:], sa[1:], w, sw, out=buf[:, 1:301])
    check(out, a[1:], sa[1:], w, sw)
    assert (buf[:, 0] == 7.0).all() and (buf[:, 301:] == 7.0).all()


def test_rows_do_not_touch_each_other():
    """A row with NaN, and a W block with an infinite scale, stay where they are."""
    rng = np.random.default_rng(6)
    a, sa = operand(20, 256, 1, rng)
    w, sw = operand(300, 256, 128, rng)
    want = lm.logits_fp8(a, sa, w, sw, out_dtype=torch.float32)
    sa2, sw2 = sa.clone(), sw.clone()
    sa2[3, 1] = float("nan")
    sw2[2, 0] = float("inf")
    got = lm.logits_fp8(a, sa2, w, sw2, out_dtype=torch.float32)
    assert got[3].isnan().all()
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[3] = False
    assert torch.equal(got[keep][:, :256], want[keep][:, :256])
    assert not torch.isfinite(got[keep][:, 256:]).any()


def test_empty_and_python_checks():
    rng = np.random.default_rng(7)
    a, sa = operand(4, 256, 1, rng)
    w, sw = operand(300, 256, 128, rng)
    assert lm.logits_fp8(a[:0], sa[:0], w, sw).shape == (0, 300)
    for bad in (lambda: lm.logits_fp8(a, sa.double(), w, sw), lambda: lm.logits_fp8(a, sa[:, :1], w, sw),
                lambda: lm.logits_fp8(a, sa, w, sw[:2]), lambda: lm.logits_fp8(a, sa, w, sw, out_dtype=torch.float16),
                lambda: lm.logits_fp8(a.float(), sa, w, sw), lambda: lm.logits_fp8(a[:, :128], sa, w, sw),
                lambda: lm.logits_fp8(a, sa, w, sw, out=torch.empty(300, 4, device="cuda").t())):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("n,vocab", [(2048, 2200), (1500, 4500), (300, 16500), (700, 1000), (64, 5000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_rows_get_equal_logits(n, vocab, dtype):
    """One hidden state at every place of the batch: the same bits everywhere."""
    rng = np.random.default_rng(n + vocab)
    hidden = 1280
    a, sa = operand(1, hidden, 1, rng)
    w, sw = operand(vocab, hidden, 128, rng)
    many = a.view(torch.uint8).expand(n, hidden).contiguous().view(torch.float8_e4m3fn)
    out = lm.logits_fp8(many, sa.expand(n, -1).contiguous(), w, sw, out_dtype=dtype)
    assert torch.equal(out, out[:1].expand_as(out)), (out != out[:1]).sum()


def test_refusals_keep_the_entry_status():
    q = torch.zeros(4, 65664, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.ones(4, 513, device="cuda")
    with pytest.raises(lm.LMHeadError) as e:
        lm.logits_fp8(q, s, q, s[:1])
    assert e.value.status == lm.LMHEAD_ERR_SHAPE


def wide_operand(rows, cols, block_rows, seed):
    """operand(), made on the device."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = (torch.randn(rows, cols, generator=g, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, torch.exp(torch.rand(-(-rows // block_rows), cols // 128, generator=g, device="cuda") * 6 - 3)


def check_wide(out, a, sa, w, sw):
    """check(), on the device: long sums of many rows and columns."""
    A = a.double() * sa.double().repeat_interleave(128, 1)
    B = w.double() * sw.double().repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)
    z = A @ B.t().contiguous()
    A.abs_(), B.abs_()
    tol = (A @ B.t().contiguous()) * ((128 + a.shape[1] // 128) * 2.0 ** -23)
    if out.dtype == torch.bfloat16:
        tol += 2.0 ** -8 * 1.01 * z.abs()
        if a.shape[0] > 64:
            for k in range(0, a.shape[1], 8):
                most = A[:, k, None] * B[None, :, k]
                for j in range(k + 1, k + 8):
                    most = torch.maximum(most, A[:, j, None] * B[None, :, j])
                tol += 8 * 2.0 ** -13 * most
    bad = ~((out.double() - z).abs() <= tol)   # NaN is bad too
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), float((out.double() - z).abs().max()))


# More columns than the stream over sets of rows takes (two groups of 16 a wave for fp32, one for bf16),
# so every one of these runs tiles: of 128 rows for n <= 128 and, with an fp32 output, wherever
# ceil(n / 128) is odd; of 256 rows for the others. 9 to 40 column blocks: the ring of four steps is
# used over and over, an odd and an even number of times.
LONG = [(70, 33001, 1280), (100, 32900, 1152), (128, 33000, 2048), (129, 22100, 1280), (200, 16500, 2048),
        (256, 16400, 4096), (300, 13101, 1152), (300, 13100, 4096), (480, 8300, 5120), (1030, 4500, 2176)]


@pytest.mark.parametrize("n,vocab,hidden", LONG)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tiles_over_long_sums(n, vocab, hidden, dtype):
    print(f"[logits] n={n} vocab={vocab} hidden={hidden} {dtype}", flush=True)
    a, sa = wide_operand(n, hidden, 1, n + hidden)
    w, sw = wide_operand(vocab, hidden, 128, vocab)
    check_wide(lm.logits_fp8(a, sa, w, sw, out_dtype=dtype), a, sa, w, sw)


# 2048 waves share the groups of 16 columns: 2, 3, 4, 5 at once, two trips of 3, 4 and 5 (shares that
# differ by a group, a last trip that is not whole), and four trips of 4
@pytest.mark.parametrize("n", [1, 16, 17, 33, 64])
@pytest.mark.parametrize("vocab,hidden", [(40000, 640), (70001, 384), (100003, 640), (151936, 256), (170000, 512),
                                          (200001, 384), (262144, 128), (310001, 256), (500009, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stream_of_many_columns(n, vocab, hidden, dtype):
    print(f"[logits] n={n} vocab={vocab} hidden={hidden} {dtype}", flush=True)
    a, sa = wide_operand(n, hidden, 1, n + hidden)
    w, sw = wide_operand(vocab, hidden, 128, vocab)
    check_wide(lm.logits_fp8(a, sa, w, sw, out_dtype=dtype), a, sa, w, sw)
