"""The operators around the projection run together, as a server or a rollout
uses them: norm -> 8-bit logits -> token, captured and replayed, on another
stream, two at once, and scored again by the log-prob entry."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm

pytestmark = pytest.mark.gpu


def setup(n, hidden, vocab, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)
    x, res = randn(n, hidden), randn(n, hidden)
    nw = 1 + randn(hidden, std=0.1)
    W = randn(vocab, hidden, std=0.1)
    u = torch.rand(n, generator=g, device="cuda").clamp(max=1 - 2.0 ** -24)
    return x, res, nw, W, u


@pytest.mark.parametrize("n", [1, 33, 300])
def test_next_token_is_its_parts_and_scores_alike(n):
    hidden, vocab = 512, 3000
    x, res, nw, W, u = setup(n, hidden, vocab, n)
    Wq, Ws = lm.quantize_fp8(W, 128)
    token, lp, r = lm.next_token(x, nw, Wq, Ws, u, residual=res, top_k=50, top_p=0.9, temperature=0.8)
    q, s, r2 = lm.rms_norm_quant(x, nw, res)
    logits = lm.logits_fp8(q, s, Wq, Ws, out_dtype=torch.float32)
    t2, lp2 = lm.sample(logits, u, temperature=0.8, top_k=50, top_p=0.9)
    assert torch.equal(token, t2) and torch.equal(lp, lp2) and torch.equal(r, r2)
    assert ((token >= 0) & (token < vocab)).all()
    # the log-prob entry on the values that the 8-bit operands stand for (bf16
    # holds q * scale to 2^-8): logits of size ~ sqrt(hidden) 0.1 ~ 2.3 move by
    # at most 2 * 2^-8 * sum |a w| / tau, with sum |a w| ~ hidden * 0.064
    A = (q.float() * s.repeat_interleave(128, 1)).to(torch.bfloat16)
    Wd = (Wq.float() * Ws.repeat_interleave(128, 0)[:vocab].repeat_interleave(128, 1)).to(torch.bfloat16)
    scored = lm.logprob(A, Wd, token, chunk=512, temperature=0.8)
    assert (scored - lp).abs().max() <= 2 * 2 * 2.0 ** -8 * hidden * 0.064 / 0.8


def test_captured_and_replayed():
    n, hidden, vocab = 5, 256, 2000
    x, res, nw, W, u = setup(n, hidden, vocab, 3)
    Wq, Ws = lm.quantize_fp8(W, 128)
    step = lambda: lm.next_token(x, nw, Wq, Ws, u, residual=res, top_p=0.9)  # noqa: E731
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
        g = torch.Generator(device="cuda")
        g.manual_seed(100 + rep)
        x.copy_(torch.randn(n, hidden, generator=g, device="cuda"))
        u.copy_(torch.rand(n, generator=g, device="cuda").clamp(max=1 - 2.0 ** -24))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_training_step_captured():
    """Forward and backward of the norm as explicit calls in a graph."""
    n, hidden = 300, 1024
    x, res, nw, W, u = setup(n, hidden, 8, 4)
    dy = torch.randn_like(x)

    def step():
        f = lm.rms_norm_forward(x, nw, res)
        dx, dw = lm.rms_norm_backward(dy, f.residual_out, nw, f.rstd, dresidual=res)
        return f.y, f.residual_out, dx, dw
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        x.normal_()
        dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), rep


def test_autograd_captured():
    """The norm's gradients through autograd in a graph, and no second derivative."""
    n, hidden = 65, 512
    x, res, nw, _, _ = setup(n, hidden, 8, 6)
    leaves = [t.clone().requires_grad_() for t in (x, res, nw)]
    dy, dr = torch.randn_like(x), torch.randn_like(x)

    def step():
        y, r = lm.rms_norm(leaves[0], leaves[2], leaves[1])
        return (y.detach(),) + torch.autograd.grad((y, r), (leaves[0], leaves[2], leaves[1]), (dy, dr))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(3):
        with torch.no_grad():
            leaves[0].normal_()
        dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), rep
    y, _ = lm.rms_norm(leaves[0], leaves[2], leaves[1])
    g, = torch.autograd.grad(y, leaves[0], dy.clone().requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_streams_at_once():
    """Two streams with their own inputs and workspaces, interleaved."""
    hidden, vocab = 512, 20000
    sets = [setup(64, hidden, vocab, s) for s in (1, 2)]
    heads = [lm.quantize_fp8(s[3], 128) for s in sets]

    def step(i):
        x, res, nw, _, u = sets[i]
        return lm.next_token(x, nw, *heads[i], u, residual=res, top_p=0.95, temperature=1.2)
    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            for a, b in zip(out, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 33, 300])
def test_next_token_scores_as_its_operands_say(n):
    """The log-prob against the 64-bit log-softmax of what the 8-bit operands
    stand for. A logit of size ~ 2.3 is 132 fp32 additions, each off by up to
    2^-23 of a partial sum, independently: some 2e-6 rms, 1.2e-5 at six sigma;
    a log-prob is a logit less a mean of them, over tau: under 1e-4."""
    hidden, vocab = 512, 3000
    x, res, nw, W, u = setup(n, hidden, vocab, n)
    Wq, Ws = lm.quantize_fp8(W, 128)
    token, lp, _ = lm.next_token(x, nw, Wq, Ws, u, residual=res, top_k=50, top_p=0.9, temperature=0.8)
    q, s, _ = lm.rms_norm_quant(x, nw, res)
    A = (q.double() * s.double().repeat_interleave(128, 1)).cpu()
    B = (Wq.double() * Ws.double().repeat_interleave(128, 0)[:vocab].repeat_interleave(128, 1)).cpu()
    want = torch.log_softmax(A @ B.t() / float(np.float32(0.8)), 1).gather(1, token.long().cpu()[:, None])[:, 0]
    assert (lp.double().cpu() - want).abs().max() <= 1e-4


def test_offsets_past_32_bits():
    """Rows, logits and draws behind the first 4 GiB: the last rows of a large
    call are those of a call on them alone."""
    def normal(rows, cols, std=1.0):
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        for r in range(0, rows, 1 << 16):
            x[r:r + (1 << 16)].normal_(0.0, std)
        return x
    print("[large] norm 1,060,000 x 4096", flush=True)
    n, hidden = 1060000, 4096
    x = normal(n, hidden)
    w = 1 + normal(1, hidden, 0.1)[0]
    f = lm.rms_norm_forward(x, w, x, out_fp8=True)
    want = lm.rms_norm_forward(x[-5:], w, x[-5:], out_fp8=True)
    for a, b in zip(f, want):
        assert torch.equal(a[-5:].view(torch.uint8), b.view(torch.uint8))
    r, rstd = f.residual_out, f.rstd
    del f
    dx, _ = lm.rms_norm_backward(x, r, w, rstd, need_dweight=False)
    assert torch.equal(dx[-5:], lm.rms_norm_backward(x[-5:], r[-5:], w, rstd[-5:], need_dweight=False)[0])
    del dx, r
    q, s = lm.quantize_fp8(x)
    q1, s1 = lm.quantize_fp8(x[-5:])
    assert torch.equal(q[-5:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-5:], s1)
    q, s = lm.quantize_fp8(x, 128)
    tail = (n - 1) // 128 * 128
    q1, s1 = lm.quantize_fp8(x[tail:], 128)
    assert torch.equal(q[tail:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-1:], s1)
    del x, q, s
    for dtype in (torch.float32, torch.bfloat16):
        print(f"[large] logits and draws 20,000 x 151,936 {dtype}", flush=True)
        n, hidden, vocab = 20000, 128, 151936
        rows = normal(1, hidden).expand(n, hidden).contiguous()
        a, sa = lm.quantize_fp8(rows)
        W, sw = lm.quantize_fp8(normal(vocab, hidden), 128)
        z = lm.logits_fp8(a, sa, W, sw, out_dtype=dtype)
        # the same hidden state in every row: its logits are those of the first
        assert torch.equal(z[-700:], z[:1].expand(700, vocab)) and torch.equal(z[9999], z[0])
        u = torch.full((n,), 0.37, device="cuda")
        token, lp = lm.sample(z, u, top_p=0.9)
        assert (token == token[0]).all() and (lp == lp[0]).all() and token[0] >= 0
        del z
