"""Binding of include/lmhead_train.h: token embedding and its gradient, the
clipped policy loss and the preference loss on log-probabilities, and the AdamW
step over many tensors.

The same two layers as the rest of the binding: the C entry points under their
own names (tensor, address or None; the status is returned), and torch helpers
that check their arguments, allocate outputs and workspace and raise
``LMHeadError``. Importable from the package itself.
"""

from __future__ import annotations

import ctypes
import functools
import operator
from typing import NamedTuple, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import LMHEAD_ERR_SHAPE, LMHeadError, _ok, _on_device_of, _p, _stream, lib
from .decode import _DTYPES, FP8_BLOCK, _check_gpu, _workspace

DTYPE_E4M3 = 2
DEVERR_TOKEN = 32

KL_K1, KL_K2, KL_K3 = 1, 2, 3
REDUCE_MEAN, REDUCE_SUM, REDUCE_SEQUENCE_MEAN = 0, 1, 2
PREFERENCE_SIGMOID, PREFERENCE_HINGE, PREFERENCE_SQUARED = 0, 1, 2

_KL = {"k1": KL_K1, "k2": KL_K2, "k3": KL_K3}
_REDUCE = {"mean": REDUCE_MEAN, "sum": REDUCE_SUM, "sequence_mean": REDUCE_SEQUENCE_MEAN}
_PREFERENCE = {"sigmoid": PREFERENCE_SIGMOID, "hinge": PREFERENCE_HINGE, "squared": PREFERENCE_SQUARED}
_WEIGHT_DTYPES = {**_DTYPES, torch.float8_e4m3fn: DTYPE_E4M3}
_WEIGHTS = tuple(_WEIGHT_DTYPES)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_BF16_F32 = (torch.bfloat16, torch.float32)


class lmhead_embedding(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("weight_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
    ]


class lmhead_policy_problem(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64),
        ("sequences", ctypes.c_int64),
        ("num_valid", ctypes.c_int64),
        ("clip_low", ctypes.c_double),
        ("clip_high", ctypes.c_double),
        ("dual_clip", ctypes.c_double),
        ("kl_weight", ctypes.c_double),
        ("kl_kind", ctypes.c_int32),
        ("reduction", ctypes.c_int32),
        ("advantage_per_sequence", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class lmhead_preference_problem(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64),
        ("pairs", ctypes.c_int64),
        ("num_pairs", ctypes.c_int64),
        ("beta", ctypes.c_double),
        ("margin", ctypes.c_double),
        ("label_smoothing", ctypes.c_double),
        ("kind", ctypes.c_int32),
        ("average", ctypes.c_int32),
    ]


class lmhead_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("exp_avg_scale", ctypes.c_void_p),
        ("exp_avg_sq_scale", ctypes.c_void_p),
        ("copy", ctypes.c_void_p),
        ("numel", ctypes.c_int64),
        ("param_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("state_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class lmhead_adamw(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
        ("step", ctypes.c_int64),
        ("device_step", ctypes.c_void_p),
        ("device_lr", ctypes.c_void_p),
        ("grad_scale", ctypes.c_void_p),
        ("stochastic", ctypes.c_int32),
        ("seed", ctypes.c_uint32),
    ]


_ready = False


def _lib() -> ctypes.CDLL:
    """The library with the argument types of this header's entries set."""
    global _ready
    L = lib()
    if not _ready:
        vp, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        E, P, F, A, T = (ctypes.POINTER(t) for t in (lmhead_embedding, lmhead_policy_problem, lmhead_preference_problem,
                                                     lmhead_adamw, lmhead_adamw_tensor))
        L.lmhead_embedding_fwd.argtypes = [E] + [vp] * 5 + [sz, vp]
        L.lmhead_embedding_bwd_workspace_size.argtypes = [E]
        L.lmhead_embedding_bwd.argtypes = [E] + [vp] * 4 + [sz, vp]
        L.lmhead_policy_loss_workspace_size.argtypes = [P]
        L.lmhead_policy_loss_fwd.argtypes = [P] + [vp] * 10 + [sz, vp]
        L.lmhead_policy_loss_bwd.argtypes = [P] + [vp] * 10
        L.lmhead_preference_loss_workspace_size.argtypes = [F]
        L.lmhead_preference_loss_fwd.argtypes = [F] + [vp] * 8 + [sz, vp]
        L.lmhead_preference_loss_bwd.argtypes = [F] + [vp] * 6
        L.lmhead_adamw_step.argtypes = [A, T, i64, vp, vp]
        L.lmhead_adamw_table_size.argtypes = [i64]
        L.lmhead_adamw_table.argtypes = [T, i64, vp, sz]
        for f in (L.lmhead_embedding_bwd_workspace_size, L.lmhead_policy_loss_workspace_size,
                  L.lmhead_preference_loss_workspace_size, L.lmhead_adamw_table_size):
            f.restype = sz
        for f in (L.lmhead_embedding_fwd, L.lmhead_embedding_bwd, L.lmhead_policy_loss_fwd, L.lmhead_policy_loss_bwd,
                  L.lmhead_preference_loss_fwd, L.lmhead_preference_loss_bwd, L.lmhead_adamw_step,
                  L.lmhead_adamw_table):
            f.restype = ctypes.c_int
        _ready = True
    return L


# ----------------------------------------------------------- C entry points

def lmhead_embedding_fwd(p, ids, weight, weight_scale, out, workspace, workspace_bytes, stream=None) -> int:
    return _lib().lmhead_embedding_fwd(ctypes.byref(p), _p(ids), _p(weight), _p(weight_scale), _p(out), _p(workspace),
                                       workspace_bytes, _stream(stream))


def lmhead_embedding_bwd_workspace_size(p) -> int:
    return int(_lib().lmhead_embedding_bwd_workspace_size(ctypes.byref(p)))


def lmhead_embedding_bwd(p, ids, dout, dweight, workspace, workspace_bytes, stream=None) -> int:
    return _lib().lmhead_embedding_bwd(ctypes.byref(p), _p(ids), _p(dout), _p(dweight), _p(workspace), workspace_bytes,
                                       _stream(stream))


def lmhead_policy_loss_workspace_size(p) -> int:
    return int(_lib().lmhead_policy_loss_workspace_size(ctypes.byref(p)))


def lmhead_policy_loss_fwd(p, logp, old_logp, ref_logp, advantage, targets, cu_seqlens, loss, stats, weights,
                           workspace, workspace_bytes, stream=None) -> int:
    return _lib().lmhead_policy_loss_fwd(ctypes.byref(p), _p(logp), _p(old_logp), _p(ref_logp), _p(advantage),
                                         _p(targets), _p(cu_seqlens), _p(loss), _p(stats), _p(weights), _p(workspace),
                                         workspace_bytes, _stream(stream))


def lmhead_policy_loss_bwd(p, grad, weights, logp, old_logp, ref_logp, advantage, targets, cu_seqlens, dlogp,
                           stream=None) -> int:
    return _lib().lmhead_policy_loss_bwd(ctypes.byref(p), _p(grad), _p(weights), _p(logp), _p(old_logp), _p(ref_logp),
                                         _p(advantage), _p(targets), _p(cu_seqlens), _p(dlogp), _stream(stream))


def lmhead_preference_loss_workspace_size(p) -> int:
    return int(_lib().lmhead_preference_loss_workspace_size(ctypes.byref(p)))


def lmhead_preference_loss_fwd(p, logp, ref_logp, targets, cu_seqlens, loss, rewards, coef, workspace,
                               workspace_bytes, stream=None) -> int:
    return _lib().lmhead_preference_loss_fwd(ctypes.byref(p), _p(logp), _p(ref_logp), _p(targets), _p(cu_seqlens),
                                             _p(loss), _p(rewards), _p(coef), _p(workspace), workspace_bytes,
                                             _stream(stream))


def lmhead_preference_loss_bwd(p, grad, coef, targets, cu_seqlens, dlogp, stream=None) -> int:
    return _lib().lmhead_preference_loss_bwd(ctypes.byref(p), _p(grad), _p(coef), _p(targets), _p(cu_seqlens),
                                             _p(dlogp), _stream(stream))


def lmhead_adamw_step(p, tensors, count, table, stream=None) -> int:
    """tensors: a ctypes array of lmhead_adamw_tensor (host), or None."""
    return _lib().lmhead_adamw_step(ctypes.byref(p), tensors, count, _p(table), _stream(stream))


def lmhead_adamw_table_size(count) -> int:
    return int(_lib().lmhead_adamw_table_size(count))


def lmhead_adamw_table(tensors, count, table, table_bytes) -> int:
    """table: a tensor in host memory, or its address."""
    return _lib().lmhead_adamw_table(tensors, count, _p(table), table_bytes)


# --------------------------------------------------------------- embedding

@_on_device_of(0)
def embedding_forward(ids, weight, scale: float = 1.0, weight_scale=None, out_dtype=None,
                      ws: Optional[torch.Tensor] = None):
    """scale * weight[ids] [n, hidden]; see lmhead_embedding_fwd. ids int32 [n],
    negative: a zero row. weight bf16 or fp32 [vocab, hidden], or e4m3 with
    weight_scale (quantize_fp8 with block_rows 128). out_dtype: the weight's
    (bf16 for e4m3) unless given. ws: 256 bytes, to read the error word."""
    _check_gpu("ids", ids, _I32, (None,))
    _check_gpu("weight", weight, _WEIGHTS, (None, None), ids.device)
    n = ids.shape[0]
    vocab, hidden = weight.shape
    if (weight_scale is not None) != (weight.dtype == torch.float8_e4m3fn):
        raise ValueError("weight_scale goes with an e4m3 weight")
    if weight_scale is not None:
        if hidden % FP8_BLOCK != 0:
            raise LMHeadError(LMHEAD_ERR_SHAPE, "lmhead_embedding_fwd")
        _check_gpu("weight_scale", weight_scale, (torch.float32,), (-(-vocab // FP8_BLOCK), hidden // FP8_BLOCK),
                   ids.device)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if weight_scale is not None else weight.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be bfloat16 or float32")
    if ws is not None:
        _check_gpu("ws", ws, (torch.uint8,), (None,), ids.device)
    p = lmhead_embedding(n, vocab, hidden, float(scale), _WEIGHT_DTYPES[weight.dtype], _DTYPES[out_dtype], 0)
    out = torch.empty(n, hidden, dtype=out_dtype, device=ids.device)
    _ok(lmhead_embedding_fwd(p, ids, weight, weight_scale, out, ws, ws.numel() if ws is not None else 0),
        "lmhead_embedding_fwd")
    return out


@_on_device_of(0)
def embedding_backward(dout, ids, vocab: int, scale: float = 1.0, out_dtype=torch.bfloat16,
                       acc: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """The gradient of embedding_forward's weight: dweight [vocab, hidden] of
    out_dtype, zeros where no token has the id; or, with acc (bf16 or fp32
    [vocab, hidden], for instance backward_accumulate's dW_acc), acc with the
    gradient added, other rows untouched. See lmhead_embedding_bwd."""
    _check_gpu("dout", dout, _BF16_F32, (None, None))
    n, hidden = dout.shape
    _check_gpu("ids", ids, _I32, (n,), dout.device)
    if acc is not None:
        _check_gpu("acc", acc, _BF16_F32, (vocab, hidden), dout.device)
        out_dtype = acc.dtype
    elif out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be bfloat16 or float32")
    p = lmhead_embedding(n, vocab, hidden, float(scale), _DTYPES[out_dtype], _DTYPES[dout.dtype], int(acc is not None))
    ws = _workspace(ws, lmhead_embedding_bwd_workspace_size(p), dout.device, lmhead_embedding_bwd, p, 4)
    dweight = torch.empty(vocab, hidden, dtype=out_dtype, device=dout.device) if acc is None else acc
    _ok(lmhead_embedding_bwd(p, ids, dout, dweight, ws, ws.numel()), "lmhead_embedding_bwd")
    return dweight


class Embedding(torch.autograd.Function):
    """Rows of a bf16 or fp32 weight by token, scaled."""

    @staticmethod
    def forward(ctx, ids, weight, scale, out_dtype):
        ctx.save_for_backward(ids)
        ctx.cfg = (weight.shape[0], scale, weight.dtype)
        return embedding_forward(ids, weight, scale, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        vocab, scale, dtype = ctx.cfg
        return None, embedding_backward(dout.contiguous(), ctx.saved_tensors[0], vocab, scale, dtype), None, None


def embedding(ids, weight, scale: float = 1.0, weight_scale=None, out_dtype=None):
    """embedding_forward with the gradient of a bf16 or fp32 weight (whole, as
    autograd adds it up; embedding_backward adds to an accumulator in place). An
    e4m3 weight has none. Differentiable once; for a backward captured into a graph
    see rms_norm."""
    if weight_scale is not None or not isinstance(weight, torch.Tensor) or weight.dtype not in _DTYPES:
        return embedding_forward(ids, weight, scale, weight_scale, out_dtype)
    return Embedding.apply(ids, weight, float(scale), out_dtype)


# ------------------------------------------------- losses on log-probabilities

class PolicyOutputs(NamedTuple):
    loss: torch.Tensor      # fp32 []
    stats: torch.Tensor     # fp32 [4]: means over counted tokens of KL, clipped, r, exp(-d) - 1 + d
    weights: torch.Tensor   # fp32 [max(sequences, 1)], for the backward


def _check_vector(name, t, dtypes, n, like):
    """A contiguous [n] of one dtype on the device of `like`; n None: any size."""
    # half the time of the general check, which says what is wrong
    if isinstance(t, torch.Tensor) and t.dtype is dtypes[0] and t.get_device() == like.get_device() and t.is_cuda and \
            t.dim() == 1 and (n is None or t.shape[0] == n) and t.is_contiguous():
        return
    _check_gpu(name, t, dtypes, (n,), like.device)


def _check_tokens(logp, targets, cu_seqlens):
    """(tokens, sequences or 0)."""
    _check_gpu("logp", logp, _F32, (None,))
    n = logp.shape[0]
    if targets is not None:
        _check_vector("targets", targets, _I32, n, logp)
    if cu_seqlens is None:
        return n, 0
    _check_vector("cu_seqlens", cu_seqlens, _I32, None, logp)
    if cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be int32 [sequences + 1], at least one sequence")
    return n, cu_seqlens.shape[0] - 1


# An output has memory of its own: views of one buffer would share its version, so
# that work in place on one (a loss divided, statistics reduced over ranks) would
# spoil the others for the backward, and one kept would keep all. new_empty of an fp32
# input is the quickest way to one.

def _scratch(ws, nbytes, like, entry, p, pointers):
    if ws is None and nbytes > 0:
        return like.new_empty(nbytes >> 2)
    return _workspace(ws, nbytes, like.device, entry, p, pointers)


def _real(x) -> float:
    """x as the C call reads it. A tensor's hash is its identity: under that a value
    changed in place would be found by its old one."""
    return x if type(x) is float else ctypes.c_double(x).value


# a problem and its workspace's size, by its numbers alone: Python's own floats and ints
@functools.lru_cache(maxsize=64)
def _policy_sizes(*numbers):
    p = lmhead_policy_problem(*numbers, 0)
    return p, lmhead_policy_loss_workspace_size(p)


@functools.lru_cache(maxsize=64)
def _preference_sizes(*numbers):
    p = lmhead_preference_problem(*numbers)
    return p, lmhead_preference_loss_workspace_size(p)


def _policy_problem(logp, advantage, old_logp, ref_logp, targets, cu_seqlens, clip_low, clip_high, dual_clip,
                    kl_weight, kl_kind, reduction, num_valid, advantage_per_sequence):
    n, sequences = _check_tokens(logp, targets, cu_seqlens)
    _check_vector("advantage", advantage, _F32, None, logp)
    per_sequence = advantage_per_sequence
    if per_sequence is None:
        if sequences == n and n > 1:
            raise ValueError("as many sequences as tokens: say by advantage_per_sequence whose advantages they are")
        per_sequence = advantage.shape[0] != n
    if (per_sequence and sequences == 0) or advantage.shape[0] != (sequences if per_sequence else n):
        raise ValueError("advantage must be float32 [n], or [sequences] with cu_seqlens")
    if old_logp is not None:
        _check_vector("old_logp", old_logp, _F32, n, logp)
    if ref_logp is not None:
        _check_vector("ref_logp", ref_logp, _F32, n, logp)
    if kl_kind not in _KL:
        raise ValueError("kl_kind must be 'k1', 'k2' or 'k3'")
    if reduction not in _REDUCE:
        raise ValueError("reduction must be 'mean', 'sum' or 'sequence_mean'")
    return _policy_sizes(n, sequences, operator.index(num_valid), _real(clip_low), _real(clip_high), _real(dual_clip),
                         _real(kl_weight), _KL[kl_kind], _REDUCE[reduction], int(per_sequence))


@_on_device_of(0)
def policy_loss_forward(logp, advantage, old_logp=None, ref_logp=None, targets=None, cu_seqlens=None,
                        clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0,
                        kl_weight: float = 0.0, kl_kind: str = "k3", reduction: str = "mean", num_valid: int = -1,
                        advantage_per_sequence: Optional[bool] = None, ws: Optional[torch.Tensor] = None) -> PolicyOutputs:
    """Clipped policy loss of packed tokens; see lmhead_policy_loss_fwd. logp fp32
    [n] (logprob's); advantage fp32 [n], or [sequences] with cu_seqlens (int32
    [sequences + 1]), told apart by its length unless advantage_per_sequence says
    which; targets int32 [n], negative: the token does not count."""
    p, nbytes = _policy_problem(logp, advantage, old_logp, ref_logp, targets, cu_seqlens, clip_low, clip_high, dual_clip,
                                kl_weight, kl_kind, reduction, num_valid, advantage_per_sequence)
    ws = _scratch(ws, nbytes, logp, lmhead_policy_loss_fwd, p, 10)
    loss, stats, weights = logp.new_empty(()), logp.new_empty(4), logp.new_empty(max(p.sequences, 1))
    _ok(lmhead_policy_loss_fwd(p, logp, old_logp, ref_logp, advantage, targets, cu_seqlens, loss, stats, weights, ws,
                               ws.numel() * ws.element_size()), "lmhead_policy_loss_fwd")
    return PolicyOutputs(loss, stats, weights)


@_on_device_of(0)
def policy_loss_backward(grad, weights, logp, advantage, old_logp=None, ref_logp=None, targets=None, cu_seqlens=None,
                         clip_low: float = 0.2, clip_high: float = 0.2, dual_clip: float = 0.0,
                         kl_weight: float = 0.0, kl_kind: str = "k3", reduction: str = "mean", num_valid: int = -1,
                         advantage_per_sequence: Optional[bool] = None):
    """dlogp fp32 [n]. grad: fp32 [1] or []; weights: the forward's; the rest as
    given to the forward."""
    p, _ = _policy_problem(logp, advantage, old_logp, ref_logp, targets, cu_seqlens, clip_low, clip_high, dual_clip,
                           kl_weight, kl_kind, reduction, num_valid, advantage_per_sequence)
    _check_scalar("grad", grad, torch.float32, logp.device)
    _check_vector("weights", weights, _F32, max(p.sequences, 1), logp)
    dlogp = torch.empty_like(logp)
    _ok(lmhead_policy_loss_bwd(p, grad, weights, logp, old_logp, ref_logp, advantage, targets, cu_seqlens, dlogp),
        "lmhead_policy_loss_bwd")
    return dlogp


def _check_scalar(name, t, dtype, device=None):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a tensor on a GPU device, that of the inputs")
    if t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name} must hold one {str(dtype).replace('torch.', '')}")


class PolicyLoss(torch.autograd.Function):
    """(loss, stats) of policy_loss_forward."""

    @staticmethod
    def forward(ctx, logp, advantage, old_logp, ref_logp, targets, cu_seqlens, how):
        f = policy_loss_forward(logp, advantage, old_logp, ref_logp, targets, cu_seqlens, *how)
        ctx.save_for_backward(f.weights, logp, advantage, old_logp, ref_logp, targets, cu_seqlens)
        ctx.how = how
        ctx.mark_non_differentiable(f.stats)
        ctx.set_materialize_grads(False)
        return f.loss, f.stats

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        if g is None:
            return (None,) * 7
        return (policy_loss_backward(g.to(torch.float32), *ctx.saved_tensors, *ctx.how),) + (None,) * 6


def policy_loss(logp, advantage, old_logp=None, ref_logp=None, targets=None, cu_seqlens=None, clip_low: float = 0.2,
                clip_high: float = 0.2, dual_clip: float = 0.0, kl_weight: float = 0.0, kl_kind: str = "k3",
                reduction: str = "mean", num_valid: int = -1, advantage_per_sequence: Optional[bool] = None):
    """(loss, stats) with the gradient of logp alone (old_logp, ref_logp and the
    advantages are constants); see policy_loss_forward. Differentiable once; for a
    backward captured into a graph see rms_norm."""
    return PolicyLoss.apply(logp, advantage, old_logp, ref_logp, targets, cu_seqlens,
                            # numbers now: the backward's are the forward's
                            (_real(clip_low), _real(clip_high), _real(dual_clip), _real(kl_weight), kl_kind, reduction,
                             operator.index(num_valid), advantage_per_sequence))


class PreferenceOutputs(NamedTuple):
    loss: torch.Tensor      # fp32 []
    rewards: torch.Tensor   # fp32 [2 pairs]: beta s of the chosen answers, then of the rejected ones
    coef: torch.Tensor      # fp32 [2 pairs], for the backward


@_on_device_of(0)
def preference_loss_forward(logp, cu_seqlens, ref_logp=None, targets=None, kind: str = "sigmoid", beta: float = 0.1,
                            margin: float = 0.0, label_smoothing: float = 0.0, average: bool = False,
                            num_pairs: int = -1, ws: Optional[torch.Tensor] = None) -> PreferenceOutputs:
    """Loss of pairs of packed answers, the chosen ones first; see
    lmhead_preference_loss_fwd. cu_seqlens int32 [2 pairs + 1]."""
    n, _ = _check_tokens(logp, targets, cu_seqlens)
    if ref_logp is not None:
        _check_vector("ref_logp", ref_logp, _F32, n, logp)
    pairs = _pairs(cu_seqlens)
    if kind not in _PREFERENCE:
        raise ValueError("kind must be 'sigmoid', 'hinge' or 'squared'")
    p, nbytes = _preference_sizes(n, pairs, operator.index(num_pairs), _real(beta), _real(margin),
                                  _real(label_smoothing), _PREFERENCE[kind], int(bool(average)))
    ws = _scratch(ws, nbytes, logp, lmhead_preference_loss_fwd, p, 8)
    loss, rewards, coef = logp.new_empty(()), logp.new_empty(2 * pairs), logp.new_empty(2 * pairs)
    _ok(lmhead_preference_loss_fwd(p, logp, ref_logp, targets, cu_seqlens, loss, rewards, coef, ws,
                                   ws.numel() * ws.element_size()), "lmhead_preference_loss_fwd")
    return PreferenceOutputs(loss, rewards, coef)


def _pairs(cu_seqlens) -> int:
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 3 or \
            cu_seqlens.shape[0] % 2 != 1:
        raise ValueError("cu_seqlens must be int32 [2 pairs + 1], at least one pair")
    return (cu_seqlens.shape[0] - 1) // 2


@_on_device_of(0)
def preference_loss_backward(grad, coef, n: int, cu_seqlens, targets=None):
    """dlogp fp32 [n]. grad: fp32 [1] or []; coef: the forward's."""
    _check_scalar("grad", grad, torch.float32)
    pairs = _pairs(cu_seqlens)
    _check_vector("cu_seqlens", cu_seqlens, _I32, None, grad)
    _check_vector("coef", coef, _F32, 2 * pairs, grad)
    if targets is not None:
        _check_vector("targets", targets, _I32, n, grad)
    p, _ = _preference_sizes(operator.index(n), pairs, -1, 1.0, 0.0, 0.0, PREFERENCE_SIGMOID, 0)
    dlogp = torch.empty(n, dtype=torch.float32, device=grad.device)
    _ok(lmhead_preference_loss_bwd(p, grad, coef, targets, cu_seqlens, dlogp), "lmhead_preference_loss_bwd")
    return dlogp


class PreferenceLoss(torch.autograd.Function):
    """(loss, rewards) of preference_loss_forward."""

    @staticmethod
    def forward(ctx, logp, cu_seqlens, ref_logp, targets, how):
        f = preference_loss_forward(logp, cu_seqlens, ref_logp, targets, *how)
        ctx.save_for_backward(f.coef, cu_seqlens, targets)
        ctx.n = logp.shape[0]
        ctx.mark_non_differentiable(f.rewards)
        ctx.set_materialize_grads(False)
        return f.loss, f.rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        if g is None:
            return (None,) * 5
        coef, cu_seqlens, targets = ctx.saved_tensors
        return (preference_loss_backward(g.to(torch.float32), coef, ctx.n, cu_seqlens, targets),) + (None,) * 4


def preference_loss(logp, cu_seqlens, ref_logp=None, targets=None, kind: str = "sigmoid", beta: float = 0.1,
                    margin: float = 0.0, label_smoothing: float = 0.0, average: bool = False, num_pairs: int = -1):
    """(loss, rewards) with the gradient of logp alone; see
    preference_loss_forward. Differentiable once; for a backward captured into a
    graph see rms_norm."""
    return PreferenceLoss.apply(logp, cu_seqlens, ref_logp, targets,
                                (kind, beta, margin, label_smoothing, average, num_pairs))


# ------------------------------------------------------------------- AdamW

class AdamWState(NamedTuple):
    exp_avg: torch.Tensor                              # fp32 or e4m3, the parameter's elements
    exp_avg_sq: torch.Tensor                           # fp32 v, or e4m3 sqrt(v)
    exp_avg_scale: Optional[torch.Tensor] = None       # e4m3: fp32 [ceil(numel / 128)]
    exp_avg_sq_scale: Optional[torch.Tensor] = None


def adamw_state(param, dtype=torch.float32) -> AdamWState:
    """A parameter's states before its first step: fp32, or float8_e4m3fn with
    block scales (2.06 bytes per element instead of 8)."""
    if dtype == torch.float32:
        return AdamWState(torch.zeros_like(param, dtype=dtype), torch.zeros_like(param, dtype=dtype))
    if dtype != torch.float8_e4m3fn:
        raise ValueError("dtype must be float32 or float8_e4m3fn")
    blocks = -(-param.numel() // FP8_BLOCK)
    m, v = (torch.zeros(param.shape, dtype=torch.uint8, device=param.device).view(dtype) for _ in range(2))
    return AdamWState(m, v, *(torch.ones(blocks, dtype=torch.float32, device=param.device) for _ in range(2)))


class AdamWPlan:
    """The tensors of a step, checked and laid out once (adamw_plan). It keeps
    the storages that the tensors had then: a parameter or gradient that is given
    another storage needs another plan. Where a gradient was its parameter's own
    .grad then, a step is refused once it no longer is (after zero_grad() without
    set_to_none=False, for instance): the plan still holds the old one. It may be
    dropped while steps are still running, on any streams; but a graph that holds a
    step reads the plan's memory: keep the plan as long as the graph."""

    def __init__(self, device, tensors, keep, own=(), watched=()):
        self.device, self.tensors, self.count, self.keep = device, tensors, len(tensors), keep
        self.own = list(own)           # (parameter, its own .grad)
        self.watched = list(watched)   # written tensors that autograd may have saved
        self.streams = set()   # that its memory is marked as in use on
        self.table = None
        if self.count > 48:   # more than a launch takes as an argument
            table = torch.empty(lmhead_adamw_table_size(self.count), dtype=torch.uint8)
            st = lmhead_adamw_table(tensors, self.count, table, table.numel())
            if st == LMHEAD_ERR_SHAPE:   # too large for one launch: without
                return
            _ok(st, "lmhead_adamw_table")
            self.table = table.to(device)
            torch.cuda.synchronize(device)   # steps may run on any stream

    def mark(self):
        """Mark the plan's memory as in use on the current stream of its device, which
        is the current one; its handle.

        The allocator hands a freed block at once to the stream that it was allocated
        on. Marked, it waits for this one first: else a plan dropped while a step
        is pending would leave the kernel another tensor's bytes for addresses. Once per
        stream: a mark holds until the block is freed. Not in a capture, whose owner
        keeps the plan."""
        stream = _stream(None)
        if stream not in self.streams and not torch.cuda.is_current_stream_capturing():
            current = torch.cuda.current_stream()
            for t in self.keep:
                t.record_stream(current)
            if self.table is not None:
                self.table.record_stream(current)
            self.streams.add(stream)
        return stream

    def step(self, p):
        """One launch of the plan's tensors on the current stream of its device,
        which is the current one."""
        for param, grad in self.own:
            if param.grad is not grad:
                at = [a is param for a, _ in self.own].index(True)
                raise ValueError(f"the .grad of parameter {at} of those planned with theirs is another tensor now: "
                                 "keep gradients in place (zero_grad(set_to_none=False)) or make another plan")
        _ok(lmhead_adamw_step(p, self.tensors, self.count, self.table, self.mark()), "lmhead_adamw_step")
        if self.watched:
            torch.autograd.graph.increment_version(self.watched)


def _check_of(i, name, t, dtypes, shape, device):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.shape == shape and t.is_contiguous() and \
            (device is None or t.get_device() == device.index):
        return
    _check_gpu(f"{name} of tensor {i}", t, dtypes, shape, device)


def adamw_plan(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], states: Sequence[AdamWState],
               copies: Optional[Sequence[Optional[torch.Tensor]]] = None) -> AdamWPlan:
    """A plan for adamw_step: parameters bf16 or fp32, gradients bf16 or fp32 of
    the same shapes (kept in place from step to step, as accumulators are),
    states from adamw_state, copies None or bf16 tensors that take the rounded
    parameters. All contiguous, on one GPU, and none sharing memory with another.
    Not while a graph is captured (the steps may be)."""
    copies = [None] * len(params) if copies is None else list(copies)
    if not len(params) == len(grads) == len(states) == len(copies):
        raise ValueError("params, grads, states and copies must be of one length")
    if len(params) == 0:
        raise ValueError("a plan needs a parameter")
    table = (lmhead_adamw_tensor * len(params))()
    dev, keep, spans, own, watched = None, [], [], [], []
    for i, (p, g, s, c) in enumerate(zip(params, grads, states, copies)):
        m, v, ms, vs = s
        shape = p.shape if isinstance(p, torch.Tensor) else ()
        _check_of(i, "params", p, _BF16_F32, shape, dev)
        dev = p.device
        _check_of(i, "grads", g, _BF16_F32, shape, dev)
        _check_of(i, "states.exp_avg", m, (torch.float32, torch.float8_e4m3fn), shape, dev)
        _check_of(i, "states.exp_avg_sq", v, (m.dtype,), shape, dev)
        e8 = m.dtype == torch.float8_e4m3fn
        if (ms is not None) != e8 or (vs is not None) != e8:
            raise ValueError(f"states[{i}]: scales go with e4m3 states")
        numel = p.numel()
        if e8:
            blocks = (-(-numel // FP8_BLOCK),)
            _check_of(i, "states.exp_avg_scale", ms, _F32, blocks, dev)
            _check_of(i, "states.exp_avg_sq_scale", vs, _F32, blocks, dev)
        if c is not None:
            _check_of(i, "copies", c, (torch.bfloat16,), shape, dev)
        at = []
        for t in (p, g, m, v, ms, vs, c):
            if t is None:
                at.append(None)
                continue
            start = t.data_ptr()
            at.append(start)
            keep.append(t.data)   # its storage now, whatever t is given later
            size = t.nbytes
            if size > 0:
                spans.append((start, start + size))
        if p.is_leaf and p.grad is g:
            own.append((p, g))
        watched += [t for t in (p, c) if t is not None and t.requires_grad]
        table[i] = (*at, numel, _DTYPES[p.dtype], _DTYPES[g.dtype], _WEIGHT_DTYPES[m.dtype], 0)
    spans.sort()
    if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
        raise ValueError("two tensors of the plan share memory")
    plan = AdamWPlan(dev, table, keep, own, watched)
    if dev.index == torch.cuda.current_device():
        plan.mark()   # here rather than in the first step: this stream's most likely
    return plan


def adamw_step(plan: AdamWPlan, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.0, grad_scale: Optional[torch.Tensor] = None,
               seed: Optional[int] = None) -> None:
    """One AdamW step of the plan's tensors, in place; see lmhead_adamw_step. A
    backward pass that saved a parameter (or copy) given to the plan as a tensor that
    requires gradients raises after the step, as after any work in place; of others
    (W.data, or at a graph's replays) autograd learns nothing: step after it.
    step: 1 for the first, or an int32 device tensor of one element (read at
    each replay of a captured step); lr: a number or an fp32 device tensor of one;
    grad_scale: an fp32 device tensor of one that multiplies the gradients. seed:
    8-bit states round at random by it, the step and the element's place, and so
    follow slow changes on average; without, to nearest."""
    p = lmhead_adamw(0.0, beta1, beta2, eps, weight_decay, 1, None, None, None, int(seed is not None),
                     (seed or 0) & 0xffffffff)
    if isinstance(step, torch.Tensor):
        _check_scalar("step", step, torch.int32, plan.device)
        p.device_step = step.data_ptr()
    else:
        p.step = int(step)
    if isinstance(lr, torch.Tensor):
        _check_scalar("lr", lr, torch.float32, plan.device)
        p.device_lr = lr.data_ptr()
    else:
        p.lr = lr
    if grad_scale is not None:
        _check_scalar("grad_scale", grad_scale, torch.float32, plan.device)
        p.grad_scale = grad_scale.data_ptr()
    if plan.device.index == torch.cuda.current_device():
        plan.step(p)
        return
    with torch.cuda.device(plan.device):
        plan.step(p)
