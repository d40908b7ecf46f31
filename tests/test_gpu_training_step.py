"""The operators around the projection run together, as a training step uses
them: ids -> embedding -> norm -> log-probs -> loss -> gradients -> one tied
matrix's accumulator -> AdamW."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Step:
    """A model of one tied matrix W and one norm: every operator once."""

    def __init__(self, n, hidden, vocab, seed, state=torch.float32):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.n, self.vocab = n, vocab
        self.W = (torch.randn(vocab, hidden, generator=g, device="cuda") * 0.05).to(BF)
        self.nw = torch.ones(hidden, dtype=BF, device="cuda")
        self.ids = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
        self.ids[::17] = -1
        self.targets = torch.randint(0, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
        self.targets[::5] = -100
        cut = torch.sort(torch.randint(0, n + 1, (7,), generator=g, device="cuda")).values
        ends = torch.tensor([0, n], device="cuda")
        self.cu = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)
        self.adv = torch.randn(8, generator=g, device="cuda")
        self.dW = torch.zeros(vocab, hidden, device="cuda")
        self.dnw = torch.zeros(hidden, dtype=BF, device="cuda")
        self.plan = lm.adamw_plan([self.W, self.nw], [self.dW, self.dnw],
                                  [lm.adamw_state(self.W, state), lm.adamw_state(self.nw)])
        self.t = torch.ones(1, dtype=torch.int32, device="cuda")
        self.one = torch.ones(1, device="cuda")

    def forward(self):
        x = lm.embedding_forward(self.ids, self.W, 2.0)
        f = lm.rms_norm_forward(x, self.nw)
        logp, lse, _ = lm.logprob_forward(f.y, self.W, self.targets, 512)
        return x, f, logp, lse

    def loss(self, logp, old, kind):
        if kind == "policy":
            args = (logp, self.adv, old, old, self.targets, self.cu)
            kw = dict(kl_weight=0.1, reduction="sequence_mean")
            f = lm.policy_loss_forward(*args, **kw)
            return f.loss, lm.policy_loss_backward(self.one, f.weights, *args, **kw)
        f = lm.preference_loss_forward(logp, self.cu, old, self.targets)
        return f.loss, lm.preference_loss_backward(self.one, f.coef, self.n, self.cu, self.targets)

    def gradients(self, old, kind):
        """Fills dW (fp32, both uses of W) and dnw; returns the loss."""
        x, f, logp, lse = self.forward()
        loss, dlogp = self.loss(logp, old, kind)
        self.dW.zero_()
        dy = torch.zeros(x.shape, device="cuda")
        dH, _ = lm.backward_accumulate(lm.ENTRY_LOGPROB, f.y, self.W, self.targets, lse, dlogp, 512,
                                       dH_acc=dy, dW_acc=self.dW, out_bf16=True)
        dx, dnw = lm.rms_norm_backward(dH, x, self.nw, f.rstd)
        self.dnw.copy_(dnw)
        lm.embedding_backward(dx, self.ids, self.vocab, scale=2.0, acc=self.dW)
        return loss

    def step(self, old, kind):
        loss = self.gradients(old, kind)
        lm.adamw_step(self.plan, self.t, 1e-2, weight_decay=0.01)
        self.t += 1
        return loss


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_gradients_are_those_of_autograd_on_the_plain_model(kind):
    """The whole chain against the same model in torch, 64 bits on the CPU."""
    s = Step(96, 128, 700, 1)
    old = s.forward()[2].clone() + 0.05 * torch.randn(96, device="cuda")
    loss = s.gradients(old, kind)
    W, nw = (t.double().cpu().requires_grad_() for t in (s.W, s.nw))
    ids, targets, cu = s.ids.cpu().long(), s.targets.cpu().long(), s.cu.cpu().tolist()
    x = torch.where((ids >= 0)[:, None], 2.0 * W[ids.clamp(min=0)], 0.0)
    y = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * nw
    z = torch.log_softmax(y @ W.t(), 1)
    valid = targets >= 0
    logp = torch.where(valid, z.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
    o = old.double().cpu()
    parts = [(a, b) for a, b in zip(cu[:-1], cu[1:])]
    if kind == "policy":
        want, adv = 0.0, s.adv.double().cpu()
        for q, (a, b) in enumerate(parts):
            at = torch.arange(a, b)[valid[a:b]]
            if len(at):
                d = logp[at] - o[at]
                r = d.exp()
                gain = torch.minimum(r * adv[q], r.clamp(0.8, 1.2) * adv[q])
                want = want + (-gain + 0.1 * (torch.expm1(-d) + d)).mean() / len(parts)
    else:
        sums = torch.stack([(logp - o)[a:b][valid[a:b]].sum() for a, b in parts])
        want = -torch.nn.functional.logsigmoid(0.1 * (sums[:4] - sums[4:])).mean()
    want.backward()
    # bf16 stands between the operators (x, y, dL/dz, dH, dx): each rounding is 2^-8 of
    # its values; through the softmax of logits of size <= |y| |w| the log-probs move by
    # at most 2^-8 sum |y w|, here a few hundredths
    dlp = 2.0 ** -8 * float((y.detach().abs() @ W.detach().abs().t()).max())
    assert abs(float(loss) - float(want.detach())) <= 4 * dlp
    # gradients as wholes: five roundings of 2^-8 in a row and the log-probs' share, which
    # changes ratios and softmax weights by dlp each
    for got, ref in ((s.dW, W.grad), (s.dnw, nw.grad)):
        off = float((got.double().cpu() - ref).norm() / ref.norm())
        assert off <= 5 * 2.0 ** -8 + 2 * dlp, off


@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_autograd_of_the_chain_gives_the_explicit_calls_gradients(kind):
    s = Step(200, 256, 1500, 2)
    old = s.forward()[2].clone()
    s.gradients(old, kind)
    W, nw = s.W.clone().requires_grad_(), s.nw.clone().requires_grad_()
    y = lm.rms_norm(lm.embedding(s.ids, W, 2.0), nw)
    logp = lm.logprob(y, W, s.targets, chunk=512)
    if kind == "policy":
        loss, _ = lm.policy_loss(logp, s.adv, old, old, s.targets, s.cu, kl_weight=0.1, reduction="sequence_mean")
    else:
        loss, _ = lm.preference_loss(logp, s.cu, old, s.targets)
    loss.backward()
    # autograd adds two bf16 gradients and rounds, the accumulator holds fp32: three half steps
    tol = 2.0 ** -8 * (3 * W.grad.abs().float() + s.dW.abs().max() * 2.0 ** -8)
    both = (W.grad.float() - s.dW).abs()
    assert (both <= tol + 2.0 ** -8 * s.dW.abs().max()).all()
    assert torch.equal(nw.grad, s.dnw)


@pytest.mark.parametrize("state", [torch.float32, torch.float8_e4m3fn])
def test_steps_repeat_and_a_captured_step_is_the_eager_one(state):
    runs = []
    for captured in (False, True):
        s = Step(300, 256, 2000, 3, state)
        old = s.forward()[2].clone()
        start = [t.clone() for t in (s.W, s.nw, *[u for u in s.plan.keep])]
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                s.step(old, "policy")
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                loss = s.step(old, "policy")
            for t, was in zip((s.W, s.nw, *s.plan.keep), start):   # the first state again
                (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).copy_(
                    was.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else was)
            s.t.fill_(1)
        losses = []
        for _ in range(4):
            if captured:
                graph.replay()
                torch.cuda.synchronize()
            else:
                loss = s.step(old, "policy")
            losses.append(loss.clone())
            s.forward()   # eager work between the replays
        runs.append([torch.stack(losses), s.W.clone(), s.nw.clone(), *[t.float() for t in s.plan.keep]])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert len(set(runs[0][0].tolist())) > 1   # the steps do move it


def test_micro_batches_of_one_mean():
    """Two halves with given counts add up to the whole batch's gradient."""
    s = Step(256, 128, 900, 4)
    x, f, logp, lse = s.forward()
    old = logp + 0.1 * torch.randn(256, device="cuda")
    adv = torch.randn(256, device="cuda")
    count = int((s.targets >= 0).sum())
    whole = lm.policy_loss_forward(logp, adv, old, targets=s.targets)
    d = lm.policy_loss_backward(s.one, whole.weights, logp, adv, old, targets=s.targets)
    loss, parts = 0.0, []
    for c in (slice(0, 100), slice(100, 256)):
        args = (logp[c], adv[c], old[c], None, s.targets[c])
        h = lm.policy_loss_forward(*args, num_valid=count)
        loss += float(h.loss)
        parts.append(lm.policy_loss_backward(s.one, h.weights, *args, num_valid=count))
    assert torch.equal(torch.cat(parts), d)
    assert abs(loss - float(whole.loss)) <= 4 * 2.0 ** -24 * float((adv.abs() * 2).mean())


def test_answer_paths_matrix_serves_the_lookup():
    """A server that holds W in 8 bits alone: embedding, norm, logits, token."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    W = (torch.randn(1000, 256, generator=g, device="cuda") * 0.1).to(BF)
    Wq, Ws = lm.quantize_fp8(W, 128)
    ids = torch.tensor([5, 999, 128], dtype=torch.int32, device="cuda")
    u = torch.rand(3, generator=g, device="cuda")
    nw = torch.ones(256, dtype=BF, device="cuda")
    for _ in range(3):
        x = lm.embedding(ids, Wq, 1.0, Ws)
        want = (Wq[ids.long()].float() * Ws[(ids // 128).long()].repeat_interleave(128, 1)).to(BF)
        assert torch.equal(x, want)
        ids, logp, _ = lm.next_token(x, nw, Wq, Ws, u)
        assert ((ids >= 0) & (ids < 1000)).all() and np.isfinite(logp.cpu().numpy()).all()
