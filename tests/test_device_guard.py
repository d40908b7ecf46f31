"""Every torch helper runs with its tensors' device current, however its first
tensor is given: on the CPU, with a stand-in for a tensor on another device."""
import contextlib
import inspect

import pytest
import torch

import chunked_lm_head_amd as lm


class Elsewhere(torch.Tensor):
    """Reports the GPU cuda:1; no data is ever read."""
    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


class Entered(Exception):
    pass


CALLS = [("ce_loss_forward", "H", 0, 4), ("logprob_forward", "H", 0, 4), ("support_forward", "H", 0, 5),
         ("support_logprob_forward", "H", 0, 4), ("support_kl_forward", "H", 0, 4), ("backward", "H", 1, 7),
         ("backward_accumulate", "H", 1, 7), ("rms_norm_forward", "x", 0, 2), ("rms_norm_backward", "dy", 0, 4),
         ("quantize_fp8", "x", 0, 1), ("logits_fp8", "a", 0, 4), ("sample", "logits", 0, 2), ("rms_norm_quant", "x", 0, 2),
         ("lmhead_read_device_error", "workspace", 0, 1)]


@pytest.fixture
def guard(monkeypatch):
    @contextlib.contextmanager
    def device(d):
        assert torch.device(d) == torch.device("cuda", 1)
        raise Entered
        yield
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    return torch.zeros(4, 128).as_subclass(Elsewhere)


@pytest.mark.parametrize("name,arg,at,count", CALLS)
def test_first_tensor_by_place_and_by_keyword(guard, name, arg, at, count):
    fn = getattr(lm, name)
    with pytest.raises(Entered):
        fn(*[guard if i == at else 1 for i in range(count)])
    names = inspect.unwrap(fn).__code__.co_varnames[:count]
    assert names[at] == arg
    with pytest.raises(Entered):
        fn(**{n: guard if n == arg else 1 for n in names})


def test_a_tensor_on_the_current_device_enters_nothing(guard, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        lm.quantize_fp8(x=guard, block_rows=7)
    with pytest.raises(ValueError):
        lm.quantize_fp8(x=torch.zeros(4, 128))
