"""The binding of include/lmhead_train.h on the host: what it hands to the entries,
with the entries and the checks for a GPU replaced."""
import numpy as np
import pytest
import torch

import chunked_lm_head_amd as lm
from chunked_lm_head_amd import train

CU = torch.tensor([0, 2, 4], dtype=torch.int32)


@pytest.fixture
def problems(monkeypatch):
    """Problems that the helpers hand to the losses' entries, as dicts."""
    seen = []

    def entry(p, *args):
        seen.append({name: getattr(p, name) for name, _ in p._fields_})
        return lm.LMHEAD_OK
    for name in ("lmhead_policy_loss_fwd", "lmhead_policy_loss_bwd", "lmhead_preference_loss_fwd",
                 "lmhead_preference_loss_bwd"):
        monkeypatch.setattr(train, name, entry)
    for name in ("_check_gpu", "_check_vector", "_check_scalar"):
        monkeypatch.setattr(train, name, lambda *a, **k: None)
    return seen


def numbers(value):
    """The same number in every form that an entry's struct takes."""
    return [torch.tensor(value, dtype=torch.float64), np.array(value), np.float64(value)]


@pytest.mark.parametrize("name", ["clip_low", "clip_high", "dual_clip", "kl_weight"])
@pytest.mark.parametrize("backward", [False, True])
def test_policy_numbers_are_read_at_each_call(problems, name, backward):
    x = torch.zeros(4)
    call = (lambda **kw: lm.policy_loss_backward(x[:1], x[:1], x, x, ref_logp=x, **kw)) if backward else \
        (lambda **kw: lm.policy_loss_forward(x, x, ref_logp=x, **kw))
    start = 2.0 if name == "dual_clip" else 0.25
    for v in numbers(start)[:2]:
        for factor in (1.0, 2.0, 2.0):
            v *= factor   # in place: the same object
            call(**{name: v})
        assert [p[name] for p in problems[-3:]] == [start, 2 * start, 4 * start]
    for v in numbers(start)[2:]:
        call(**{name: v})
        assert problems[-1][name] == start


@pytest.mark.parametrize("name", ["beta", "margin", "label_smoothing"])
def test_preference_numbers_are_read_at_each_call(problems, name):
    x = torch.zeros(4)
    for v in numbers(0.125)[:2]:
        for factor in (1.0, 2.0, 2.0):
            v *= factor
            lm.preference_loss_forward(x, CU, **{name: v})
        assert [p[name] for p in problems[-3:]] == [0.125, 0.25, 0.5]


@pytest.mark.parametrize("count", [torch.tensor(3), np.int64(3), np.array(3), 3])
def test_given_counts_are_read_at_each_call(problems, count):
    x = torch.zeros(4)
    for want in (3, 5):
        lm.policy_loss_forward(x, x, num_valid=count)
        assert problems[-1]["num_valid"] == want
        lm.preference_loss_forward(x, CU, num_pairs=count)
        assert problems[-1]["num_pairs"] == want
        count += 2


def test_a_backward_takes_the_forwards_numbers(problems, monkeypatch):
    x, k = torch.zeros(4, requires_grad=True), torch.tensor(0.25)
    loss, _ = lm.policy_loss(x, x.detach(), ref_logp=x.detach(), kl_weight=k)
    k.mul_(2)
    loss.backward()
    assert [p["kl_weight"] for p in problems] == [0.25, 0.25]
    scales = []

    def entry(p, *args):
        scales.append(p.scale)
        return lm.LMHEAD_OK
    monkeypatch.setattr(train, "lmhead_embedding_fwd", entry)
    monkeypatch.setattr(train, "lmhead_embedding_bwd", entry)
    w, k = torch.zeros(5, 64, requires_grad=True), torch.tensor(0.25)
    y = lm.embedding(torch.zeros(3, dtype=torch.int32), w, k)
    k.mul_(2)
    y.backward(torch.zeros_like(y))
    assert scales == [0.25, 0.25]


def test_what_is_no_number_is_refused(problems):
    x = torch.zeros(4)
    for bad in ("0.1", None, torch.zeros(2), [0.1]):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            lm.policy_loss_forward(x, x, clip_low=bad)
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            lm.preference_loss_forward(x, CU, beta=bad)
    for bad in ("3", 1.5, torch.tensor(1.5)):
        with pytest.raises(TypeError):
            lm.policy_loss_forward(x, x, num_valid=bad)
        with pytest.raises(TypeError):
            lm.preference_loss_forward(x, CU, num_pairs=bad)
    assert not problems


def divided(loss, other):
    loss /= 4


def added(loss, other):
    loss += 1.0


def reduced(loss, other):
    other.mul_(2)


def detached(loss, other):
    loss.detach().mul_(0)


@pytest.mark.parametrize("how,factor", [(divided, 0.25), (added, 1.0), (reduced, 1.0), (detached, 1.0)])
@pytest.mark.parametrize("kind", ["policy", "preference"])
def test_outputs_may_be_worked_on_in_place(problems, monkeypatch, kind, how, factor):
    """Before the backward, as programs do for logs and for accumulated batches."""
    grads = []
    for name in ("lmhead_policy_loss_bwd", "lmhead_preference_loss_bwd"):
        monkeypatch.setattr(train, name, lambda p, grad, *args: grads.append(float(grad)) or lm.LMHEAD_OK)
    x = torch.zeros(4, requires_grad=True)
    loss, other = lm.policy_loss(x, x.detach(), cu_seqlens=CU, advantage_per_sequence=False) if kind == "policy" else \
        lm.preference_loss(x, CU)
    how(loss, other)
    loss.backward()
    assert grads == [factor] and x.grad.shape == (4,)


def test_outputs_keep_no_others_memory(problems):
    x = torch.zeros(4)
    for f in (lm.policy_loss_forward(x, x), lm.preference_loss_forward(x, CU)):
        for t in f:
            assert t._base is None and t.untyped_storage().nbytes() == 4 * t.numel()


def test_the_cross_entropys_loss_may_be_worked_on_in_place(monkeypatch):
    grads = []
    monkeypatch.setattr(lm, "_check_inputs", lambda *a, **k: None)
    monkeypatch.setattr(lm, "workspace", lambda *a: torch.empty(256, dtype=torch.uint8))
    monkeypatch.setattr(lm, "lmhead_loss_fwd", lambda *a: lm.LMHEAD_OK)
    monkeypatch.setattr(lm, "backward", lambda entry, H, W, targets, lse, grad, *a, **k:
                        grads.append(grad.tolist()) or (torch.zeros_like(H), torch.zeros_like(W)))
    H, W = torch.zeros(4, 64, requires_grad=True), torch.zeros(9, 64, requires_grad=True)
    loss = lm.ChunkedLMHeadCE.apply(H, W, torch.zeros(4, dtype=torch.int32), 256)
    assert loss.shape == ()
    loss /= 4
    loss.backward()
    assert grads == [[0.25]]


class Marked:
    """Stands for a tensor of a plan."""

    def __init__(self):
        self.on = []

    def record_stream(self, stream):
        self.on.append(stream)


def test_a_plans_memory_is_marked_on_every_stream_that_steps(monkeypatch):
    """Read by a kernel on another stream than its own, a block must not go back to
    its own before: the plan may be dropped while the step is pending."""
    now = dict(stream=0, capturing=False)
    launched = []

    def entry(p, tensors, count, table, stream=None):
        launched.append(train._stream(stream))
        return lm.LMHEAD_OK
    monkeypatch.setattr(train, "lmhead_adamw_step", entry)
    monkeypatch.setattr(train, "_stream", lambda s: now["stream"] if s is None else s)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    keep = [Marked(), Marked()]
    plan = lm.AdamWPlan(torch.device("cuda", 0), (lm.lmhead_adamw_tensor * 2)(), keep)
    plan.table = Marked()
    all_ = keep + [plan.table]
    for stream, marks in ((0, [0]), (0, [0]), (7, [0, 7]), (0, [0, 7]), (7, [0, 7])):
        now["stream"] = stream
        lm.adamw_step(plan, 1, 0.1)
        assert [m.on for m in all_] == [marks] * 3 and launched[-1] == stream
    # a capture only records its launch; the graph's owner keeps the plan. The stream's first eager step marks
    now.update(stream=9, capturing=True)
    lm.adamw_step(plan, 1, 0.1)
    assert [m.on for m in all_] == [[0, 7]] * 3 and launched[-1] == 9
    now["capturing"] = False
    lm.adamw_step(plan, 1, 0.1)
    assert [m.on for m in all_] == [[0, 7, 9]] * 3


@pytest.fixture
def host_plan(monkeypatch):
    """adamw_plan of CPU tensors, its steps counted instead of launched."""
    steps = []
    monkeypatch.setattr(train, "_check_of", lambda *a: None)
    monkeypatch.setattr(train, "lmhead_adamw_step", lambda *a: steps.append(1) or lm.LMHEAD_OK)
    monkeypatch.setattr(train, "_stream", lambda s: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)

    def make(*args):
        plan = lm.adamw_plan(*args)
        plan.device = torch.device("cuda", 0)
        return plan
    make.steps = steps
    return make


def leaf(n=4):
    return torch.ones(n, requires_grad=True)


def test_a_replaced_gradient_is_refused(host_plan):
    a, b = leaf(), leaf()
    acc = torch.zeros(4)
    (a.sum() + b.sum()).backward()
    plan = host_plan([a, b], [acc, b.grad], [lm.adamw_state(a), lm.adamw_state(b)])   # a's is an accumulator elsewhere
    opt = torch.optim.SGD([a, b], lr=0.1)
    lm.adamw_step(plan, 1, 0.1)
    opt.zero_grad(set_to_none=False)
    (2 * b).sum().backward()
    a.grad = None
    lm.adamw_step(plan, 2, 0.1)
    assert len(host_plan.steps) == 2
    opt.zero_grad()
    with pytest.raises(ValueError, match="set_to_none"):
        lm.adamw_step(plan, 3, 0.1)
    b.sum().backward()
    with pytest.raises(ValueError, match="set_to_none"):
        lm.adamw_step(plan, 3, 0.1)
    assert len(host_plan.steps) == 2
    lm.adamw_step(host_plan([b], [b.grad], [lm.adamw_state(b)]), 3, 0.1)
    assert len(host_plan.steps) == 3


def test_a_backward_that_saved_a_parameter_raises_after_the_step(host_plan):
    w, master, frozen = leaf(), torch.ones(4), torch.ones(4)
    copy = torch.ones(4, dtype=torch.bfloat16, requires_grad=True)
    plan = host_plan([w, master, frozen], [torch.zeros(4) for _ in range(3)],
                     [lm.adamw_state(t) for t in (w, master, frozen)], [None, copy, None])
    for t in (w, copy):
        y = (t * t).sum()
        lm.adamw_step(plan, 1, 0.1)
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            y.backward()
        y = (t * t).sum()
        y.backward()
    before = frozen._version
    lm.adamw_step(plan, 2, 0.1)
    assert frozen._version == before
