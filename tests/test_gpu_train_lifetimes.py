"""Lifetimes of what the training step's operators read: plans dropped while steps
are pending, on other streams than their memory's own."""
import pytest
import torch

import chunked_lm_head_amd as lm

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_a_plan_dropped_while_its_step_is_pending():
    """The table of 60 tensors, made on one stream, read on another behind work that
    takes a while: its block comes back to the first stream only after that. Nothing
    here writes to what is allocated meanwhile."""
    count, numel = 60, 5000
    own, other = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(8192, 8192, device="cuda").to(BF)
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        ps, ds = ([torch.ones(numel, device="cuda") for _ in range(count)] for _ in range(2))
        plan = lm.adamw_plan(ps, ds, [lm.adamw_state(p) for p in ps])
        size, table = plan.table.numel(), plan.table.data_ptr()
        later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]   # no new segment later
        del later
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(40):   # some 30 ms
            torch.mm(a, a, out=b)
        lm.adamw_step(plan, 1, 0.5)
        done = torch.cuda.Event()
        done.record()
    del plan
    with torch.cuda.stream(own):
        later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    pending = not done.query()
    assert pending, "the work in front of the step was too short to show anything"
    assert table not in [t.data_ptr() for t in later]
    torch.cuda.synchronize()
    # the first step moves by lr against the gradient's sign
    assert all(((p - 0.5).abs() < 1e-6).all() for p in ps)
    with torch.cuda.stream(own):   # then it does
        later += [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()


def test_states_that_only_a_plan_keeps():
    """States made and dropped on one stream, stepped on another."""
    own, other = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(8192, 8192, device="cuda").to(BF)
    b = torch.empty_like(a)
    p, d = torch.ones(1 << 20, device="cuda"), torch.ones(1 << 20, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(own):
        state = lm.adamw_state(p)
        plan = lm.adamw_plan([p], [d], [state])
        at = [t.data_ptr() for t in state[:2]]
        del state
        later = [torch.empty(1 << 20, device="cuda") for _ in range(6)]
        del later
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(40):
            torch.mm(a, a, out=b)
        lm.adamw_step(plan, 1, 0.5)
        done = torch.cuda.Event()
        done.record()
    del plan
    with torch.cuda.stream(own):
        later = [torch.empty(1 << 20, device="cuda") for _ in range(6)]
    assert not done.query()
    assert not set(at) & {t.data_ptr() for t in later}
    torch.cuda.synchronize()
    assert ((p - 0.5).abs() < 1e-6).all()


def test_a_training_loop_through_autograd():
    """ids -> embedding -> norm -> log-probs -> policy loss, accumulated over two
    micro-batches, then a step of a plan of the parameters with their own gradients:
    what the loop gives is what a fresh plan of copies gives from the same gradients."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    n, hidden, vocab = 120, 128, 400
    W = (torch.randn(vocab, hidden, generator=g, device="cuda") * 0.1).to(BF).requires_grad_()
    nw = torch.ones(hidden, dtype=BF, device="cuda").requires_grad_()
    states = [lm.adamw_state(W, torch.float8_e4m3fn), lm.adamw_state(nw)]
    plan = None
    opt = torch.optim.SGD([W, nw], lr=0.0)   # for its zero_grad
    kl = torch.tensor(0.1)

    def loss_of():
        ids = torch.randint(-1, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
        targets = torch.randint(-100, vocab, (n,), generator=g, device="cuda", dtype=torch.int32)
        adv = torch.randn(n, generator=g, device="cuda")
        logp = lm.logprob(lm.rms_norm(lm.embedding(ids, W), nw), W, targets, chunk=256)
        loss, stats = lm.policy_loss(logp, adv, logp.detach() - 0.1, logp.detach() + 0.1, targets, kl_weight=kl)
        stats.mul_(0.5)
        loss /= 2
        return loss
    for t in range(1, 4):
        for _ in range(2):
            loss_of().backward()
        kl.mul_(0.5)
        if plan is None:
            plan = lm.adamw_plan([W, nw], [W.grad, nw.grad], states)
        twins = [x.detach().clone() for x in (W, nw)]
        copies = [lm.AdamWState(*[None if x is None else (x.view(torch.uint8).clone().view(x.dtype)
                                                          if x.dtype == torch.float8_e4m3fn else x.clone()) for x in s])
                  for s in states]
        late = loss_of()
        lm.adamw_step(plan, t, 1e-2, weight_decay=0.1, seed=t)
        lm.adamw_step(lm.adamw_plan(twins, [W.grad.clone(), nw.grad.clone()], copies), t, 1e-2, weight_decay=0.1, seed=t)
        assert torch.equal(W, twins[0]) and torch.equal(nw, twins[1])
        assert all(torch.equal(a.float(), b.float()) for s, c in zip(states, copies) for a, b in zip(s, c) if a is not None)
        with pytest.raises(RuntimeError, match="modified by an inplace"):   # its W is gone
            late.backward()
        opt.zero_grad(set_to_none=False)
        assert (W.grad == 0).all()
    opt.zero_grad()
    loss_of().backward()
    was = W.detach().clone()
    with pytest.raises(ValueError, match="set_to_none"):
        lm.adamw_step(plan, 4, 1e-2)
    assert torch.equal(W, was)
