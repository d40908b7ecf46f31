"""Token embedding and its gradient against the plain 64-bit definitions."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import train_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}   # half a step of the type, relative


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def token_ids(n, vocab, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        ids = rng.integers(0, vocab, n)
    elif kind == "one":
        ids = np.full(n, vocab // 2)
    elif kind == "sorted":
        ids = np.sort(rng.integers(0, max(1, vocab // 3), n))
    elif kind == "bucket":   # ids of one bucket only: equal low bits
        ids = rng.integers(0, vocab, n) // 2048 * 2048
    else:                    # a few common ones, padding
        ids = np.where(rng.random(n) < 0.6, rng.integers(0, min(3, vocab), n), rng.integers(0, vocab, n))
        ids = np.where(rng.random(n) < 0.1, -100, ids)
    return torch.from_numpy(ids.astype(np.int32)).cuda()


@pytest.mark.parametrize("n,vocab,hidden", [(1, 1, 64), (1, 1000, 4096), (3, 50, 192), (17, 300, 512), (200, 5000, 2112),
                                            (5, 40, 65536), (1031, 129, 64), (64, 700, 4160)])
@pytest.mark.parametrize("weight", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
def test_rows(n, vocab, hidden, weight, out):
    g = gen(n + hidden)
    ids, w = token_ids(n, vocab, "mixed", n), randn(g, vocab, hidden, dtype=weight)
    for scale in (1.0, 12.5):
        got = f64(lm.embedding_forward(ids, w, scale=scale, out_dtype=out))
        want = ref.embedding(ids.cpu().numpy(), f64(w), scale)
        # the fp32 product, then the type
        assert (np.abs(got - want) <= (2.0 ** -24 + HALF[out] * 1.0001) * np.abs(want)).all()
    if weight == out:   # no scale: the very bits
        assert np.array_equal(f64(lm.embedding(ids, w)), ref.embedding(ids.cpu().numpy(), f64(w), 1.0))


@pytest.mark.parametrize("n,vocab,hidden", [(1, 128, 128), (9, 1, 128), (300, 1000, 640), (70, 4000, 4096), (3, 200, 65536)])
@pytest.mark.parametrize("out", [BF, F32])
def test_rows_of_an_8_bit_matrix(n, vocab, hidden, out):
    g = gen(n)
    q, s = lm.quantize_fp8(randn(g, vocab, hidden, std=0.02), 128)
    ids = token_ids(n, vocab, "mixed", n)
    w = f64(q.float()) * np.repeat(np.repeat(f64(s), 128, 0)[:vocab], 128, 1)
    got = f64(lm.embedding(ids, q, 3.0, s, out))
    want = ref.embedding(ids.cpu().numpy(), w, 3.0)
    # value times block scale, times scale, then the type
    assert (np.abs(got - want) <= (2 * 2.0 ** -24 + HALF[out] * 1.0001) * np.abs(want)).all()


def test_ids_past_the_vocabulary():
    g = gen(5)
    w, ws = randn(g, 100, 256), torch.zeros(256, dtype=torch.uint8, device="cuda")
    ids = torch.tensor([3, 99, -1, 100, 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    out = lm.embedding_forward(ids, w, ws=ws)
    assert lm.lmhead_read_device_error(ws) == (lm.DEVERR_TOKEN, 3)
    assert torch.equal(out[[0, 1, 4]], w[[3, 99, 7]]) and (out[[2, 6]] == 0).all() and out[[3, 5]].isnan().all()
    lm.embedding_forward(ids[:3], w, ws=ws)
    assert lm.lmhead_read_device_error(ws) == (0, -1)
    lm.embedding_forward(ids, w, ws=ws)
    lm.embedding_forward(ids[:0], w, ws=ws)
    assert lm.lmhead_read_device_error(ws) == (0, -1)
    # the gradient leaves them out and says so
    p = lm.lmhead_embedding(7, 100, 256, 1.0, 1, 0, 0)
    ws = torch.empty(lm.lmhead_embedding_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    dout = randn(g, 7, 256)
    dw = lm.embedding_backward(dout, ids, 100, out_dtype=F32, ws=ws)
    assert lm.lmhead_read_device_error(ws) == (lm.DEVERR_TOKEN, 3)
    want = torch.zeros(100, 256, device="cuda")
    want[[3, 99, 7]] = dout[[0, 1, 4]].float()
    assert torch.equal(dw, want)
    lm.embedding_backward(dout[:3], ids[:3], 100, ws=ws)
    assert lm.lmhead_read_device_error(ws) == (0, -1)


def check_grad(ids, dout, vocab, scale, got, old, before):
    s, a, c = ref.embedding_grad(ids.cpu().numpy(), f64(dout), vocab, scale)
    want = s + (before if old else 0.0)
    got64 = f64(got)
    # c terms: at most c additions and one product, each off by 2^-24 of sums no
    # larger than that of the magnitudes; then one addition and one rounding
    tol = a * (c[:, None] + 2) * 2.0 ** -24 * 1.01 + np.abs(want) * (HALF[got.dtype] * 1.0001 + 2.0 ** -24)
    assert (np.abs(got64 - want) <= tol).all(), np.abs(got64 - want).max()
    none = c == 0
    assert np.array_equal(got64[none], (before if old else np.zeros_like(want))[none])


SHAPES = [(1, 1, 64), (31, 40, 64), (32, 2, 128), (33, 2, 128), (64, 9000, 512), (65, 700, 2112), (777, 5000, 256),
          (100, 30, 8192), (3001, 20000, 128)]


@pytest.mark.parametrize("n,vocab,hidden", SHAPES)
@pytest.mark.parametrize("kind", ["uniform", "one", "sorted", "bucket", "mixed"])
def test_gradient(n, vocab, hidden, kind):
    g = gen(n + vocab)
    ids = token_ids(n, vocab, kind, n + hidden)
    for dout_type, into in ((BF, BF), (BF, F32), (F32, F32), (F32, BF)):
        dout = randn(g, n, hidden, dtype=dout_type)
        got = lm.embedding_backward(dout, ids, vocab, scale=3.0, out_dtype=into)
        check_grad(ids, dout, vocab, 3.0, got, False, None)
        assert torch.equal(got, lm.embedding_backward(dout, ids, vocab, scale=3.0, out_dtype=into))
        acc = randn(g, vocab, hidden, dtype=into)
        before = f64(acc)
        assert lm.embedding_backward(dout, ids, vocab, scale=0.5, acc=acc) is acc
        check_grad(ids, dout, vocab, 0.5, acc, True, before)


def test_gradient_of_nothing():
    none = torch.empty(0, 256, dtype=BF, device="cuda")
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    assert (lm.embedding_backward(none, ids, 1000) == 0).all()
    assert (lm.embedding_backward(none, ids, 70001, out_dtype=F32) == 0).all()
    acc = torch.full((1000, 256), float("nan"), device="cuda")
    lm.embedding_backward(none, ids, 1000, acc=acc)
    assert acc.isnan().all()
    pad = torch.full((40,), -1, dtype=torch.int32, device="cuda")
    dout = torch.full((40, 256), float("nan"), dtype=BF, device="cuda")
    assert (lm.embedding_backward(dout, pad, 1000) == 0).all()
    lm.embedding_backward(dout, pad, 1000, acc=acc.zero_())
    assert (acc == 0).all()
    assert lm.embedding_forward(ids, torch.ones(3, 64, device="cuda")).shape == (0, 64)


def test_untouched_rows_and_padding_stay_apart():
    """NaN in rows that no token has, and in gradients of padded places, stays there."""
    g = gen(8)
    ids = torch.tensor([4, -1, 9, 4], dtype=torch.int32, device="cuda")
    dout = randn(g, 4, 128)
    dout[1] = float("nan")
    acc = torch.full((20, 128), float("nan"), device="cuda")
    acc[4] = acc[9] = 1.0
    lm.embedding_backward(dout, ids, 20, acc=acc)
    assert torch.equal(acc[9], 1.0 + dout[2].float()) and acc[4].isfinite().all()
    assert acc[[i for i in range(20) if i not in (4, 9)]].isnan().all()


def test_long_runs_pass_many_blocks():
    """One id over 2^15 tokens, and two that meet inside a block."""
    n, hidden, vocab = 1 << 15, 320, 1000
    g = gen(9)
    dout = randn(g, n, hidden)
    ids = torch.full((n,), 17, dtype=torch.int32, device="cuda")
    ids[n // 2 + 5:] = 17 + 512
    got = lm.embedding_backward(dout, ids, vocab, out_dtype=F32)
    d = dout.double()
    for v, part in ((17, d[:n // 2 + 5]), (17 + 512, d[n // 2 + 5:])):
        # the longest chain of additions: 32 of a block, 1024 / 16 / 2 of a wave, 17 of the waves
        tol = (32 + 32 + 17 + 2) * 2.0 ** -24 * part.abs().sum(0)
        assert ((got[v].double() - part.sum(0)).abs() <= tol).all()
    assert (got.abs().sum(1) != 0).sum() == 2


def test_tables_past_4_gib():
    vocab, hidden = 540000, 4096   # 4.4 GB of bf16
    w = torch.zeros(vocab, hidden, dtype=BF, device="cuda")
    ids = torch.tensor([vocab - 1, 0, 524288, vocab - 1, 524287], dtype=torch.int32, device="cuda")
    g = gen(3)
    rows = randn(g, 5, hidden)
    for i in range(5):
        w[ids[i]] = rows[i]
    want = torch.stack([w[v] for v in ids.tolist()])
    assert torch.equal(lm.embedding_forward(ids, w), want)
    dout = randn(g, 5, hidden)
    got = lm.embedding_backward(dout, ids, vocab, acc=w)
    assert got is w
    for i, v in ((1, 0), (2, 524288), (4, 524287)):
        assert torch.equal(w[v].float(), (want[i].float() + dout[i].float()).to(BF).float())
    both = want[0].float() + (dout[0].float() + dout[3].float())
    assert torch.equal(w[vocab - 1], both.to(BF))
    w.fill_(1.0)
    dense = lm.embedding_backward(dout, ids, vocab)
    assert torch.equal(dense[524288], dout[2]) and int((dense != 0).any(1).sum()) == 4


def test_many_tokens_past_4_gib():
    n, hidden, vocab = 540000, 4096, 300   # dout of 4.4 GB
    g = gen(4)
    dout = torch.zeros(n, hidden, dtype=BF, device="cuda")
    last = randn(g, hidden)
    dout[-1] = last
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    ids[-1] = 299
    got = lm.embedding_backward(dout, ids, vocab, out_dtype=F32)
    assert torch.equal(got[299], last.float()) and int((got != 0).any(1).sum()) == 1
    out = lm.embedding_forward(ids, got.to(BF))
    assert torch.equal(out[-1], last) and int((out != 0).any(1).sum()) == 1


def test_autograd():
    g = gen(6)
    vocab, hidden, n = 50, 128, 30
    ids = token_ids(n, vocab, "mixed", 3)
    for dtype in (BF, F32):
        w = randn(g, vocab, hidden, dtype=dtype).requires_grad_()
        dout = randn(g, n, hidden, dtype=dtype)
        y = lm.embedding(ids, w, 2.0)
        y.backward(dout)
        assert torch.equal(w.grad, lm.embedding_backward(dout, ids, vocab, 2.0, dtype))
        with pytest.raises(RuntimeError):
            (gw,) = torch.autograd.grad(lm.embedding(ids, w, 2.0).sum(), w, create_graph=True)
            gw.sum().backward()
    # an expanded upstream gradient
    w = randn(g, vocab, hidden).requires_grad_()
    lm.embedding(ids, w).sum().backward()
    assert torch.equal(w.grad, lm.embedding_backward(torch.ones(n, hidden, dtype=BF, device="cuda"), ids, vocab))


def test_captured_and_replayed_with_eager_work_between():
    n, vocab, hidden = 500, 3000, 256
    g = gen(7)
    w, dout, acc = randn(g, vocab, hidden), randn(g, n, hidden), torch.zeros(vocab, hidden, device="cuda")
    ids = token_ids(n, vocab, "mixed", 1)

    def step():
        acc.zero_()
        lm.embedding_backward(dout, ids, vocab, acc=acc)
        return lm.embedding_forward(ids, w, 2.0), lm.embedding_backward(dout, ids, vocab), acc.clone()
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
        ids.copy_(token_ids(n, vocab, ["uniform", "one", "mixed", "sorted"][rep], rep))
        dout.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), rep


def test_two_streams_at_once():
    n, vocab, hidden = 4000, 20000, 512
    g = gen(11)
    dout = [randn(g, n, hidden) for _ in range(2)]
    ids = [token_ids(n, vocab, "mixed", i) for i in range(2)]
    want = [lm.embedding_backward(d, i, vocab) for d, i in zip(dout, ids)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        got = []
        for s, d, i in zip(streams, dout, ids):
            with torch.cuda.stream(s):
                got.append(lm.embedding_backward(d, i, vocab))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_the_helpers():
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.zeros(10, 128, dtype=BF, device="cuda")
    q = torch.zeros(10, 128, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.ones(1, 1, device="cuda")
    for call in (lambda: lm.embedding(ids.long(), w), lambda: lm.embedding(ids.view(2, 2), w),
                 lambda: lm.embedding(ids[::2], w), lambda: lm.embedding(ids, w.t()), lambda: lm.embedding(ids, w.half()),
                 lambda: lm.embedding(ids, q), lambda: lm.embedding(ids, w, weight_scale=s),
                 lambda: lm.embedding(ids, q, weight_scale=s.repeat(2, 1)), lambda: lm.embedding(ids, w, out_dtype=torch.half),
                 lambda: lm.embedding_backward(w[:4], ids, 10, out_dtype=torch.half),
                 lambda: lm.embedding_backward(w[:3], ids, 10),
                 lambda: lm.embedding_backward(w[:4], ids, 10, acc=w[:9]),
                 lambda: lm.embedding_forward(ids, w, ws=s)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lm.embedding(ids, w[:, :100].contiguous()), lambda: lm.embedding(ids, w, float("inf")),
                 lambda: lm.embedding_backward(w[:4], ids, 0), lambda: lm.embedding(ids, q[:, :64].contiguous(), 1.0, s)):
        with pytest.raises(lm.LMHeadError):
            call()
    odd = torch.zeros(11 * 128 + 1, dtype=BF, device="cuda")[1:1 + 1280].view(10, 128)
    with pytest.raises(lm.LMHeadError):   # not 16-byte aligned
        lm.embedding(ids, odd)
