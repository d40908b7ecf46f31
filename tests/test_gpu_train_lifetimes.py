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
