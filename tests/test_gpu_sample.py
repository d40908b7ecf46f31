"""Sampling against the 64-bit rule: tokens equal, log-probabilities to half an
fp32 step plus what integer weights of 2^-44 leave (under 1e-8)."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
import decode_ref as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(v, dtype=torch.float32):
    return torch.from_numpy(np.asarray(v)).to(dtype).cuda()


def check(logits, u, **kw):
    """Filters as numbers or numpy arrays; compares with the definition."""
    n = logits.shape[0]
    args = {k: (dev(v, torch.int32 if k == "top_k" else torch.float32) if isinstance(v, np.ndarray) else v)
            for k, v in kw.items()}
    token, lp = lm.sample(logits, u, **args)
    # what the kernel is given: fp32 values of the filters
    val = {k: (f64(a) if isinstance(a, torch.Tensor) else np.float64(np.float32(a))) for k, a in args.items()}
    want, wlp = ref.sample(f64(logits), f64(u), val.get("temperature"), val.get("top_k"), val.get("top_p"),
                           val.get("min_p"))
    got = token.cpu().numpy()
    assert np.array_equal(got, want), (n, np.argwhere(got != want)[:4].ravel(), got[got != want][:4],
                                       want[got != want][:4])
    assert (np.abs(f64(lp) - wlp) <= 2.0 ** -24 * 1.01 * np.abs(wlp) + 1e-8).all()
    return token, lp


def logits_of(n, vocab, dtype, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((spread * rng.standard_normal((n, vocab))).astype(np.float32)).to(dtype).cuda()
    u = torch.from_numpy(rng.random(n).astype(np.float32)).clamp(max=1 - 2.0 ** -24).cuda()
    return x, u, rng


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=5), dict(top_k=50, top_p=0.9, temperature=0.8),
           dict(top_p=0.95), dict(top_p=0.3), dict(min_p=0.05), dict(min_p=1.0), dict(top_p=0.9, min_p=0.02, top_k=1000),
           dict(top_p=1e-6), dict(top_k=100000, top_p=0.999999), dict(temperature=3.0, top_p=0.5)]


@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 64, 65, 257, 1000, 4099, 33333])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_filters(vocab, dtype):
    x, u, _ = logits_of(9, vocab, dtype, vocab)
    for kw in FILTERS:
        print(f"[sample] vocab={vocab} {dtype} {kw}", flush=True)
        check(x, u, **kw)


@pytest.mark.parametrize("n,vocab", [(1, 151936), (70, 5000), (300, 1000), (2, 300000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_with_their_own_filters(n, vocab, dtype):
    x, u, rng = logits_of(n, vocab, dtype, n + vocab, 1.3)
    check(x, u, temperature=rng.uniform(0.3, 2.0, n).astype(np.float32),
          top_k=rng.choice([-3, 0, 1, 7, 200, vocab, 1 << 30], n).astype(np.int32),
          top_p=rng.choice([1.0, 0.5, 0.9, 0.99], n).astype(np.float32),
          min_p=rng.choice([0.0, 0.01, 0.3], n).astype(np.float32))
    check(x, u, top_p=0.95)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_logits_go_to_the_lowest_index(dtype):
    n, vocab = 40, 3001
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.integers(-2, 3, (n, vocab)).astype(np.float32)).to(dtype).cuda()
    x[1] = 0.0
    x[2, ::2] = -0.0            # -0 and +0 are equal
    x[2, 1::2] = 0.0
    x[3] = -3.0
    u = torch.from_numpy(rng.random(n).astype(np.float32)).clamp(max=1 - 2.0 ** -24).cuda()
    for kw in (dict(), dict(top_k=1), dict(top_k=10), dict(top_k=700), dict(top_k=1500, top_p=0.75), dict(top_p=0.5),
               dict(top_p=0.999), dict(min_p=0.5), dict(min_p=1.0), dict(top_p=0.25, min_p=0.9)):
        check(x, u, **kw)
    assert lm.sample(x[1:2], u[:1], top_k=1)[0].item() == 0
    # u at both ends: the first kept token, and the last
    ends = torch.tensor([0.0, 1 - 2.0 ** -24], device="cuda")
    t, _ = lm.sample(x[1:2].expand(2, vocab).contiguous(), ends, top_k=100)
    assert t.tolist() == [0, 99]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab,values", [(1500, 2), (5000, 7), (20000, 3), (40000, 1), (70000, 40)])
def test_borders_among_many_equal_logits(dtype, vocab, values):
    """From some hundred to all tokens tied where the filters end: borders that
    are listed and sorted, and more of them than the list holds."""
    n = 12
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.integers(0, values, (n, vocab)).astype(np.float32) / 4).to(dtype).cuda()
    x[3, ::3] = float("-inf")
    u = torch.from_numpy(rng.random(n).astype(np.float32)).clamp(max=1 - 2.0 ** -24).cuda()
    for kw in (dict(), dict(top_k=vocab // 3), dict(top_p=0.4), dict(top_p=0.97), dict(min_p=0.7),
               dict(top_k=vocab // 2, top_p=0.6), dict(top_k=vocab - vocab // 9, top_p=0.9, min_p=0.3)):
        print(f"[sample] vocab={vocab} values={values} {dtype} {kw}", flush=True)
        check(x, u, **kw)


def test_weights_that_vanish():
    """Temperatures so low that most weights are 0: filters that would reach into
    those, and a range of logits wider than weights can tell apart."""
    x, u, rng = logits_of(16, 30000, torch.float32, 21, 5.0)
    x[5, 100:] -= 1e30
    x[6, 1:] = -3e38
    for t in (0.01, 0.1, 1e-30):
        for kw in (dict(), dict(top_k=50), dict(top_k=20000), dict(top_p=0.999999), dict(min_p=1e-30),
                   dict(top_k=9000, top_p=0.5, min_p=1e-12)):
            check(x, u, temperature=t, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_min_p_at_the_smallest_integer_weights(dtype):
    """min-p compares integers of 2^-44; u = 0 draws the first token that is kept."""
    order = float(np.log(2.0))
    x = torch.linspace(-47 * order, 0, 4000, dtype=torch.float64).flip(0)
    x = torch.cat([x, x.flip(0)]).to(dtype)     # 0 down to 47 orders and up again
    w = np.round(np.exp2(44 + f64(x) / order))
    for first in (3300, 3500, 3700, 3730, 3760, 3800, 3990):   # the row begins about there, goes down, then up
        row, v = x[first:], w[first:]
        for min_p in (2.0 ** -44, 1.01 * 2.0 ** -44, 1.5 * 2.0 ** -44, 2.0 ** -43, 3.3 * 2.0 ** -44, 1e-13, 1e-12, 1e-30):
            floor = np.ceil(float(np.float32(min_p)) * 2.0 ** 44)
            kept = np.flatnonzero((v >= floor) & (v > 0))
            token, _ = lm.sample(row[None].cuda(), torch.zeros(1, device="cuda"), min_p=min_p)
            assert int(token) == kept[0], (first, min_p, int(token), kept[0])


def test_a_range_past_the_largest_float():
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.uniform(-3.3e38, 3.3e38, (20, 3000)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random(20).astype(np.float32)).clamp(max=1 - 2.0 ** -24).cuda()
    for kw in (dict(min_p=0.01), dict(min_p=0.04), dict(min_p=0.2), dict(top_p=0.9), dict(top_k=2000, min_p=0.045),
               dict(top_k=2900, top_p=0.999), dict()):
        check(x, u, temperature=2e38, **kw)


def test_more_rows_than_one_set_of_launches():
    x, u, rng = logits_of(700, 300, torch.bfloat16, 22)
    x[600, 5] = float("nan")
    ws = torch.empty(lm.lmhead_sample_workspace_size(lm.lmhead_sample_problem(700, 300, 300, 0)), dtype=torch.uint8,
                     device="cuda")
    token, _ = lm.sample(x, u, top_k=20, top_p=0.8, ws=ws)
    assert lm.lmhead_read_device_error(ws) == (lm.DEVERR_LOGIT, 600) and token[600] == -1
    x[600, 5] = 0.0
    check(x, u, top_k=rng.integers(0, 40, 700).astype(np.int32), top_p=0.8)


def test_masks():
    n, vocab = 12, 2500
    x, u, rng = logits_of(n, vocab, torch.float32, 8)
    x[0] = float("-inf")                         # nothing left
    x[1] = float("-inf")
    x[1, 77] = -3.0                              # one token left
    x[2, :2499] = float("-inf")
    x[3, 5:] = float("-inf")
    x[4] = torch.finfo(torch.float32).min        # the type's lowest value is a number
    x[5, 10:] = torch.finfo(torch.float32).min
    x[6] = torch.where(torch.rand(vocab, device="cuda") < 0.99, torch.tensor(float("-inf"), device="cuda"), x[6])
    x[7, :1000] = float("-inf")
    x[8] = 3.0e38
    x[8, ::3] = -3.0e38
    for kw in (dict(), dict(top_k=3), dict(top_k=64), dict(top_p=0.9), dict(min_p=0.1, top_p=0.5, top_k=600)):
        token, lp = check(x, u, **kw)
        assert token[0] == -1 and lp[0] == 0 and token[1] == 77 and lp[1] == 0 and token[2] == 2499
    # the lowest value of bf16
    xb = x.to(torch.bfloat16)
    xb[4] = torch.finfo(torch.bfloat16).min
    check(xb, u, top_p=0.9)


def test_bad_rows_and_the_error_word():
    n, vocab = 9, 700
    x, u, _ = logits_of(n, vocab, torch.float32, 9)
    clean, clean_lp = lm.sample(x, u, top_p=0.9)
    x[2, 600] = float("nan")
    x[3, 0] = float("inf")
    u2 = u.clone()
    u2[4], u2[5], u2[6] = 1.0, float("nan"), -0.1
    ws = torch.empty(lm.lmhead_sample_workspace_size(lm.lmhead_sample_problem(n, vocab, vocab, 1)), dtype=torch.uint8,
                     device="cuda")
    token, lp = lm.sample(x, u2, top_p=0.9, ws=ws)
    bad = torch.tensor([2, 3, 4, 5, 6], device="cuda")
    assert (token[bad] == -1).all() and lp[bad].isnan().all()
    rest = torch.tensor([0, 1, 7, 8], device="cuda")
    assert torch.equal(token[rest], clean[rest]) and torch.equal(lp[rest], clean_lp[rest])
    assert lm.lmhead_read_device_error(ws) == (lm.DEVERR_LOGIT | lm.DEVERR_SAMPLING, 2)
    lm.sample(x[:2], u[:2], ws=ws)
    assert lm.lmhead_read_device_error(ws) == (0, -1)
    ones = torch.ones(n, device="cuda")
    for name, values in (("temperature", [0.0, -1.0, float("nan"), float("inf")]), ("top_p", [0.0, 1.5, float("nan")]),
                         ("min_p", [-0.1, 1.5, float("nan")])):
        for v in values:
            rows = ones.clone()
            rows[8] = v
            token, lp = lm.sample(x, u, ws=ws, **{name: rows})
            assert token[8] == -1 and lp[8].isnan()
            code = lm.lmhead_read_device_error(ws)[0]
            assert code & (lm.DEVERR_TEMPERATURE if name == "temperature" else lm.DEVERR_SAMPLING)
            assert token[0] >= 0


def test_row_strides_and_offsets():
    """Rows at any element: the neighbours' values never reach a row."""
    rng = np.random.default_rng(10)
    for dtype in (torch.float32, torch.bfloat16):
        for vocab, ld in ((1000, 1001), (777, 777), (33, 36), (2047, 2100)):
            buf = torch.full((6, ld), float("nan"), dtype=dtype, device="cuda")
            buf[:, :vocab] = torch.from_numpy(rng.standard_normal((6, vocab)).astype(np.float32)).to(dtype)
            u = torch.from_numpy(rng.random(6).astype(np.float32)).clamp(max=1 - 2.0 ** -24).cuda()
            x = buf[:, :vocab]
            got = lm.sample(x, u, top_k=20, top_p=0.9)
            want = lm.sample(x.contiguous(), u, top_k=20, top_p=0.9)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            check(x, u, top_p=0.8)


def test_scalar_and_row_filters_agree():
    x, u, _ = logits_of(20, 3000, torch.float32, 12)
    full = torch.full((20,), 1.0, device="cuda")
    a = lm.sample(x, u, temperature=0.8, top_k=40, top_p=0.9, min_p=0.01)
    b = lm.sample(x, u, temperature=full * 0.8, top_k=torch.full((20,), 40, dtype=torch.int32, device="cuda"),
                  top_p=full * 0.9, min_p=full * 0.01)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert lm.sample(x, u, want_logprob=False)[1] is None
    assert torch.equal(lm.sample(x, u, want_logprob=False, top_p=0.7)[0], lm.sample(x, u, top_p=0.7)[0])


def test_draws_follow_the_distribution():
    """4096 evenly spaced u over one row: the counts are the probabilities to one
    count per token (each token's interval holds floor or ceil of its share)."""
    vocab, n = 50, 4096
    rng = np.random.default_rng(14)
    row = rng.standard_normal(vocab)
    x = dev(row).expand(n, vocab).contiguous()
    u = (torch.arange(n, device="cuda", dtype=torch.float32) + 0.5) / n
    token, _ = lm.sample(x, u)
    p = np.exp(f64(x[0]) - f64(x[0]).max())
    p /= p.sum()
    counts = np.bincount(token.cpu().numpy(), minlength=vocab)
    assert (np.abs(counts - n * p) <= 1.0 + 1e-6).all()


def test_python_checks():
    x, u, _ = logits_of(3, 100, torch.float32, 15)
    for bad in (lambda: lm.sample(x.half(), u), lambda: lm.sample(x, u[:2]), lambda: lm.sample(x, u.double()),
                lambda: lm.sample(x.t(), u), lambda: lm.sample(x, u, temperature=0.0), lambda: lm.sample(x, u, top_p=0.0),
                lambda: lm.sample(x, u, top_k=torch.ones(3, device="cuda")), lambda: lm.sample(x, u, min_p=u[:1]),
                lambda: lm.sample(x, u, temperature=1e-50), lambda: lm.sample(x, u, top_p=1e-50),
                lambda: lm.sample(x, u, top_k=(1 << 32) + 5), lambda: lm.sample(x, u, top_k=2.5),
                lambda: lm.sample(x[0], u), lambda: lm.sample(x[:1].expand(3, 100), u)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lm.LMHeadError):
        lm.sample(x, u, top_k=-2)
    t, lp = lm.sample(x[:0], u[:0])
    assert t.shape == (0,) and lp.shape == (0,)


@pytest.mark.parametrize("vocab,dtype,below", [(1 << 20, torch.float32, 28.0), (1 << 22, torch.float32, 28.5),
                                               (1 << 22, torch.bfloat16, 27.75), (3000001, torch.float32, 28.1),
                                               (1 << 26, torch.bfloat16, 26.0)])
def test_logprob_of_vocabularies_beyond_the_integers(vocab, dtype, below):
    """Millions of tokens near or below half of the integer weights' step: the
    log-probability counts what they weigh, whatever the filters."""
    x = torch.full((2, vocab), -below, dtype=dtype, device="cuda")
    x[0, 12345] = 0.0
    x[1, :5] = 0.0
    x[1, 5::7] = float("-inf")
    u = torch.tensor([0.3, 0.7], device="cuda")
    v = float(x[0, 0])
    left = vocab - 5 - len(range(5, vocab, 7))
    want = -np.log(np.array([1 + (vocab - 1) * np.exp(v), 5 + left * np.exp(v)]))
    for kw in (dict(), dict(top_k=3), dict(top_p=0.9), dict(min_p=0.5), dict(top_k=vocab // 2, top_p=0.5)):
        token, lp = lm.sample(x, u, **kw)
        assert token[0] == 12345 and token[1] < 5
        assert (np.abs(f64(lp) - want) <= 2.0 ** -24 * 1.01 * np.abs(want) + 1e-8).all(), (kw, f64(lp) - want)


def test_refusals_keep_the_entry_status():
    x, u, _ = logits_of(3, 100, torch.float32, 15)
    for kw in (dict(top_p=1.5), dict(min_p=float("nan")), dict(min_p=-0.5), dict(top_k=-2), dict(temperature=float("inf"))):
        with pytest.raises(lm.LMHeadError) as e:
            lm.sample(x, u, **kw)
        assert e.value.status == lm.LMHEAD_ERR_ARG, kw
