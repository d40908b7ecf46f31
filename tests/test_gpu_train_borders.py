"""The training step's operators on both sides of each border between launch shapes:
widths of the single launch, tiles and their joins, pieces of runs."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import test_gpu_embedding as te
import test_gpu_token_losses as tl
import train_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24

# 512 tokens: the single launch's width; 4096 tokens, 64 sequences: its end; 1024: a tile, and the sequences
# that one workgroup joins
LOSS_SIZES = [(511, 7), (512, 7), (513, 7), (1024, 9), (1025, 9), (2048, 12), (4095, 64), (4096, 64), (4097, 64),
              (4096, 65), (600, 64), (600, 66), (5120, 130), (6000, 1024), (6000, 1025)]


@pytest.mark.parametrize("n,sequences", LOSS_SIZES)
@pytest.mark.parametrize("kind", ["even", "empty", "skewed"])
@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
def test_policy(n, sequences, kind, reduction):
    tl.test_policy(n, sequences, kind, reduction)


@pytest.mark.parametrize("n,pairs", [(n, -(-s // 2)) for n, s in LOSS_SIZES] + [(9000, 1024), (9000, 1025)])
@pytest.mark.parametrize("kind", ["even", "empty", "skewed"])
@pytest.mark.parametrize("how", [dict(label_smoothing=0.2), dict(kind="squared", beta=0.5, average=True)])
def test_preference(n, pairs, kind, how):
    tl.test_preference(n, pairs, kind, how)


@pytest.mark.parametrize("tiles", [8192, 8193])
def test_losses_of_many_tiles(tiles):
    """8 tiles per thread of the joining workgroup: above, sequences' and pairs' parts
    are added by workgroups of their own. Whole numbers and powers of two, so that
    sums are exact and every output has one right value."""
    n, sequences = tiles * 1024 - 5, 6
    g = torch.Generator(device="cuda")
    g.manual_seed(tiles)
    cu = torch.tensor([0, 1, 5000, n // 2, n // 2, n - 7, n - 3], dtype=torch.int32, device="cuda")
    adv = torch.randint(-8, 9, (n,), generator=g, device="cuda").float()
    logp = torch.zeros(n, device="cuda")
    f = lm.policy_loss_forward(logp, adv, cu_seqlens=cu, reduction="sequence_mean")
    ends = cu.tolist()
    means = [float(adv[a:b].double().mean()) if b > a else 0.0 for a, b in zip(ends, ends[1:])]
    want = -sum(means) / sequences
    assert abs(float(f.loss) - want) <= 2 * U * abs(want) + 1e-15 * n
    w = f.weights.double().cpu().numpy()
    full = np.array([1.0 / (sequences * (b - a)) if b > a else 0.0 for a, b in zip(ends, ends[1:])])
    assert (np.abs(w - full) <= U * full * 1.01).all()
    d = lm.policy_loss_backward(torch.ones(1, device="cuda"), f.weights, logp, adv, cu_seqlens=cu,
                                reduction="sequence_mean")
    for s, (a, b) in enumerate(zip(ends, ends[1:])):
        assert torch.equal(d[a:b], f.weights[s] * -adv[a:b])
    assert (d[n - 3:] == 0).all()
    f = lm.policy_loss_forward(logp, adv, cu_seqlens=cu, reduction="sum")
    assert float(f.loss) == float(np.float32(-adv[:n - 3].double().sum().item()))
    # answers whose sums are whole numbers
    f = lm.preference_loss_forward(adv, cu, beta=1.0, kind="squared")
    s = np.array([float(adv[a:b].double().sum()) for a, b in zip(ends, ends[1:])])
    h = s[:3] - s[3:]
    assert f.rewards.double().tolist() == s.astype(np.float32).tolist()
    want = ((h - 0.5) ** 2).mean()
    assert abs(float(f.loss) - want) <= 2 * U * want
    slope = (2 * (h - 0.5) / 3).astype(np.float32)
    coef = f.coef.cpu().numpy()
    assert (np.abs(coef[:3] - slope) <= 2 * U * np.abs(slope)).all() and (coef[3:] == -coef[:3]).all()


# 8192 tokens: pieces of 16 up to there, of 64 above; 131,072 ids: twice as many buckets above. Hidden 1024: two
# parts of a row
@pytest.mark.parametrize("n,vocab,hidden", [(16, 40, 64), (17, 40, 64), (8191, 300, 128), (8192, 300, 1024),
                                            (8193, 300, 1024), (9001, 300, 1088), (9001, 8, 64), (20000, 700, 576),
                                            (9001, 131072, 64), (9001, 131073, 64)])
@pytest.mark.parametrize("kind", ["uniform", "one", "sorted", "mixed"])
def test_gradient(n, vocab, hidden, kind):
    g = te.gen(n + vocab)
    ids = te.token_ids(n, vocab, kind, n + hidden)
    for dout_type, into in ((BF, BF), (BF, F32), (F32, F32), (F32, BF)):
        dout = te.randn(g, n, hidden, dtype=dout_type)
        got = lm.embedding_backward(dout, ids, vocab, scale=3.0, out_dtype=into)
        te.check_grad(ids, dout, vocab, 3.0, got, False, None)
        assert torch.equal(got, lm.embedding_backward(dout, ids, vocab, scale=3.0, out_dtype=into))
        acc = te.randn(g, vocab, hidden, dtype=into)
        before = te.f64(acc)
        assert lm.embedding_backward(dout, ids, vocab, scale=0.5, acc=acc) is acc
        te.check_grad(ids, dout, vocab, 0.5, acc, True, before)


@pytest.mark.parametrize("into", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_runs_of_one_to_three_pieces(into, accumulate):
    """Runs of 1 .. 200 tokens above 8192 tokens, every id its own number of them."""
    lengths = np.concatenate([np.arange(1, 201)] * 2)
    ids = np.repeat(np.arange(400), lengths)
    np.random.default_rng(0).shuffle(ids)
    n, vocab, hidden = len(ids), 400, 192
    assert n > 8192
    g = te.gen(1)
    ids = torch.from_numpy(ids.astype(np.int32)).cuda()
    dout = te.randn(g, n, hidden)
    acc = te.randn(g, vocab, hidden, dtype=into) if accumulate else None
    before = te.f64(acc) if accumulate else None
    got = lm.embedding_backward(dout, ids, vocab, out_dtype=into, acc=acc)
    te.check_grad(ids, dout, vocab, 1.0, got, accumulate, before)


def test_the_longest_chain_of_additions():
    """Two ids over 2^15 tokens. A sum's longest chain: 64 tokens of a piece; of its 257
    pieces every eighth one, 33, by a wave; 8 waves."""
    n, hidden, vocab = 1 << 15, 320, 1000
    g = te.gen(9)
    dout = te.randn(g, n, hidden)
    cut = n // 2 + 5
    ids = torch.full((n,), 17, dtype=torch.int32, device="cuda")
    ids[cut:] = 17 + 512
    got = lm.embedding_backward(dout, ids, vocab, out_dtype=F32)
    assert -(-cut // 64) == 257
    d = dout.double()
    for v, part in ((17, d[:cut]), (17 + 512, d[cut:])):
        tol = (64 + 33 + 8) * U * part.abs().sum(0)
        assert ((got[v].double() - part.sum(0)).abs() <= tol).all()
    assert (got.abs().sum(1) != 0).sum() == 2


@pytest.mark.parametrize("weight", [BF, F32, torch.float8_e4m3fn])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("less", [0, 1])
def test_rows_on_both_sides_of_the_caches(weight, out, less):
    """64 MB of output: past the caches from there on. Rows times a power of two: the very bits."""
    hidden, vocab = 2048, 3000
    n = (64 << 20) // (hidden * (2 if out == BF else 4)) - less
    g = te.gen(n)
    w, scale = te.randn(g, vocab, hidden, dtype=F32 if weight == F32 else BF), None
    ids = torch.randint(-200, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
    at = ids.clamp(min=0).long()
    if weight == torch.float8_e4m3fn:
        w, scale = lm.quantize_fp8(w, 128)
        rows = w.float()[at] * scale[at // 128].repeat_interleave(128, 1)
    else:
        rows = w[at].float()
    want = torch.where((ids >= 0)[:, None], rows * 4.0, 0.0).to(out)
    assert torch.equal(lm.embedding_forward(ids, w, 4.0, scale, out), want)
