"""Binding of include/lmhead_decode.h: the final RMS norm (forward, backward,
8-bit output), the block quantiser, 8-bit logits and next-token sampling.

The same two layers as the rest of the binding: the C entry points under their
own names (tensor, address or None; the status is returned), and torch helpers
that check their arguments, allocate outputs and workspace and raise
``LMHeadError``. Importable from the package itself.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import (LMHEAD_ERR_SHAPE, LMHeadError, _check_f32, _ok, _on_device_of, _p, _stream, lib)

DTYPE_BF16 = 0
DTYPE_F32 = 1

DEVERR_LOGIT = 8
DEVERR_SAMPLING = 16

FP8_BLOCK = 128

_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


class lmhead_norm(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("weight_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class lmhead_fp8_problem(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("hidden", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("out_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class lmhead_sample_problem(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("logits_dtype", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("temperature", ctypes.c_float),
        ("top_p", ctypes.c_float),
        ("min_p", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("row_temperature", ctypes.c_void_p),
        ("row_top_k", ctypes.c_void_p),
        ("row_top_p", ctypes.c_void_p),
        ("row_min_p", ctypes.c_void_p),
    ]


_ready = False


def _lib() -> ctypes.CDLL:
    """The library with the argument types of this header's entries set."""
    global _ready
    L = lib()
    if not _ready:
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        N, F, S = (ctypes.POINTER(t) for t in (lmhead_norm, lmhead_fp8_problem, lmhead_sample_problem))
        L.lmhead_rms_norm_fwd.argtypes = [N] + [vp] * 9
        L.lmhead_rms_norm_bwd_workspace_size.argtypes = [N]
        L.lmhead_rms_norm_bwd.argtypes = [N] + [vp] * 8 + [sz, vp]
        L.lmhead_quantize_fp8.argtypes = [i64, i64, i32, vp, vp, vp, vp]
        L.lmhead_logits_fp8_workspace_size.argtypes = [F]
        L.lmhead_logits_fp8.argtypes = [F] + [vp] * 6 + [sz, vp]
        L.lmhead_sample_workspace_size.argtypes = [S]
        L.lmhead_sample.argtypes = [S] + [vp] * 5 + [sz, vp]
        for f in (L.lmhead_rms_norm_bwd_workspace_size, L.lmhead_logits_fp8_workspace_size,
                  L.lmhead_sample_workspace_size):
            f.restype = sz
        for f in (L.lmhead_rms_norm_fwd, L.lmhead_rms_norm_bwd, L.lmhead_quantize_fp8, L.lmhead_logits_fp8,
                  L.lmhead_sample):
            f.restype = ctypes.c_int
        _ready = True
    return L


# ----------------------------------------------------------- C entry points

def lmhead_rms_norm_fwd(p, x, residual, weight, residual_out, y, q, scale, rstd, stream=None) -> int:
    return _lib().lmhead_rms_norm_fwd(ctypes.byref(p), _p(x), _p(residual), _p(weight), _p(residual_out),
                                      _p(y), _p(q), _p(scale), _p(rstd), _stream(stream))


def lmhead_rms_norm_bwd_workspace_size(p) -> int:
    return int(_lib().lmhead_rms_norm_bwd_workspace_size(ctypes.byref(p)))


def lmhead_rms_norm_bwd(p, dy, r, weight, rstd, dresidual, dx, dweight, workspace, workspace_bytes,
                        stream=None) -> int:
    return _lib().lmhead_rms_norm_bwd(ctypes.byref(p), _p(dy), _p(r), _p(weight), _p(rstd), _p(dresidual),
                                      _p(dx), _p(dweight), _p(workspace), workspace_bytes, _stream(stream))


def lmhead_quantize_fp8(rows, cols, block_rows, x, q, scale, stream=None) -> int:
    return _lib().lmhead_quantize_fp8(rows, cols, block_rows, _p(x), _p(q), _p(scale), _stream(stream))


def lmhead_logits_fp8_workspace_size(p) -> int:
    return int(_lib().lmhead_logits_fp8_workspace_size(ctypes.byref(p)))


def lmhead_logits_fp8(p, a, a_scale, w, w_scale, out, workspace, workspace_bytes, stream=None) -> int:
    return _lib().lmhead_logits_fp8(ctypes.byref(p), _p(a), _p(a_scale), _p(w), _p(w_scale), _p(out),
                                    _p(workspace), workspace_bytes, _stream(stream))


def lmhead_sample_workspace_size(p) -> int:
    return int(_lib().lmhead_sample_workspace_size(ctypes.byref(p)))


def lmhead_sample(p, logits, u, token, logprob, workspace, workspace_bytes, stream=None) -> int:
    return _lib().lmhead_sample(ctypes.byref(p), _p(logits), _p(u), _p(token), _p(logprob), _p(workspace),
                                workspace_bytes, _stream(stream))


# ------------------------------------------------------------- torch helpers

def _check_gpu(name, t, dtypes, shape, device=None):
    """A contiguous GPU tensor of one of the dtypes; None in shape: any size."""
    # a call on one row is over in a few microseconds: the good case first, the reasons after
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous() and \
            (device is None or t.device == device):
        got = t.shape
        if len(got) == len(shape):
            for want, have in zip(shape, got):
                if want is not None and want != have:
                    break
            else:
                return
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on the inputs' device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d).replace('torch.', '') for d in dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have the shape {['any' if w is None else w for w in shape]}")


def _workspace(ws: Optional[torch.Tensor], nbytes: int, device, entry, p, pointers: int) -> torch.Tensor:
    if nbytes == 0:   # an invalid problem: the entry, which checks that first, says why
        raise LMHeadError(entry(p, *[None] * pointers, 0, stream=0), entry.__name__)
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    _check_gpu("ws", ws, (torch.uint8,), (None,), device)
    return ws


class NormOutputs(NamedTuple):
    y: Optional[torch.Tensor]              # bf16 [n, hidden]
    residual_out: Optional[torch.Tensor]   # bf16 [n, hidden], with a residual
    rstd: Optional[torch.Tensor]           # fp32 [n]
    q: Optional[torch.Tensor]              # e4m3 [n, hidden]
    scale: Optional[torch.Tensor]          # fp32 [n, hidden / 128]


def _norm_problem(x, weight, eps, weight_offset):
    _check_gpu("x", x, (torch.bfloat16,), (None, None))
    _check_gpu("weight", weight, (torch.bfloat16, torch.float32), (x.shape[1],), x.device)
    return lmhead_norm(x.shape[0], x.shape[1], float(eps), float(weight_offset), _DTYPES[weight.dtype], 0)


@_on_device_of(0)
def rms_norm_forward(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0,
                     out_bf16: bool = True, out_fp8: bool = False, out_rstd: bool = True) -> NormOutputs:
    """RMS norm of the rows of x (+ residual): see lmhead_rms_norm_fwd. out_fp8
    adds the 8-bit output with its scales, out_bf16=False leaves y out,
    out_rstd=False what only the backward needs."""
    p = _norm_problem(x, weight, eps, weight_offset)
    n, hidden = x.shape
    dev = x.device
    r = None
    if residual is not None:
        _check_gpu("residual", residual, (torch.bfloat16,), (n, hidden), dev)
        r = torch.empty_like(x)
    if out_fp8 and hidden % FP8_BLOCK != 0:
        raise LMHeadError(LMHEAD_ERR_SHAPE, "lmhead_rms_norm_fwd")
    y = torch.empty_like(x) if out_bf16 else None
    q = torch.empty(n, hidden, dtype=torch.float8_e4m3fn, device=dev) if out_fp8 else None
    scale = torch.empty(n, hidden // FP8_BLOCK, dtype=torch.float32, device=dev) if out_fp8 else None
    rstd = torch.empty(n, dtype=torch.float32, device=dev) if out_rstd else None
    _ok(lmhead_rms_norm_fwd(p, x, residual, weight, r, y, q, scale, rstd), "lmhead_rms_norm_fwd")
    return NormOutputs(y, r, rstd, q, scale)


def rms_norm_quant(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """The norm's 8-bit output for logits_fp8: (q e4m3 [n, hidden], scale fp32
    [n, hidden / 128], residual_out or None)."""
    f = rms_norm_forward(x, weight, residual, eps, weight_offset, out_bf16=False, out_fp8=True, out_rstd=False)
    return f.q, f.scale, f.residual_out


@_on_device_of(0)
def rms_norm_backward(dy, r, weight, rstd, dresidual=None, weight_offset: float = 0.0,
                      need_dx: bool = True, need_dweight: bool = True, ws: Optional[torch.Tensor] = None):
    """Returns (dx bf16 [n, hidden] or None, dweight [hidden] of the weight's
    type or None). r: the forward's residual_out, or its x without a residual."""
    p = _norm_problem(r, weight, 0.0, weight_offset)
    n, hidden = r.shape
    _check_gpu("dy", dy, (torch.bfloat16,), (n, hidden), r.device)
    _check_f32("rstd", rstd, (n,), r.device, required=n > 0)
    if dresidual is not None:
        _check_gpu("dresidual", dresidual, (torch.bfloat16,), (n, hidden), r.device)
    dx = torch.empty_like(r) if need_dx else None
    dw = torch.empty_like(weight) if need_dweight else None
    if need_dweight:
        ws = _workspace(ws, lmhead_rms_norm_bwd_workspace_size(p), r.device, lmhead_rms_norm_bwd, p, 8)
    _ok(lmhead_rms_norm_bwd(p, dy, r, weight, rstd, dresidual, dx, dw, ws, ws.numel() if ws is not None else 0),
        "lmhead_rms_norm_bwd")
    return dx, dw


class RMSNorm(torch.autograd.Function):
    """y of lmhead_rms_norm_fwd, and the new residual stream where there is one."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, weight_offset):
        f = rms_norm_forward(x, weight, residual, eps, weight_offset)
        ctx.save_for_backward(x if residual is None else f.residual_out, weight, f.rstd)
        ctx.weight_offset = weight_offset
        ctx.set_materialize_grads(False)
        return (f.y, f.residual_out) if residual is not None else f.y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr=None):
        r, weight, rstd = ctx.saved_tensors
        need_x, need_w, need_res = ctx.needs_input_grad[:3]
        if dy is None:   # only the residual stream was used
            return (dr if need_x else None), None, (dr if need_res else None), None, None
        dx, dw = rms_norm_backward(dy.contiguous(), r, weight, rstd, None if dr is None else dr.contiguous(),
                                   ctx.weight_offset, need_dx=need_x or need_res, need_dweight=need_w)
        return (dx if need_x else None), dw, (dx if need_res else None), None, None


def rms_norm(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """RMS norm with gradients for x, weight and residual: y, or (y, residual_out)
    with a residual. weight_offset 1 for zero-centred weights. Differentiable once.
    A backward captured into a graph must be the leaves' only one: drop eager
    graphs of the same leaves first (torch's gradient accumulation ties a leaf
    to the stream of its first use), or take torch.autograd.grad."""
    return RMSNorm.apply(x, weight, residual, eps, weight_offset)


@_on_device_of(0)
def quantize_fp8(x, block_rows: int = 1):
    """bf16 [rows, cols] to (q e4m3 [rows, cols], scale fp32 [ceil(rows /
    block_rows), cols / 128]); block_rows 1 for hidden states, 128 for W."""
    _check_gpu("x", x, (torch.bfloat16,), (None, None))
    rows, cols = x.shape
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError("block_rows must be 1 or 128")
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(-(-rows // block_rows), cols // FP8_BLOCK, dtype=torch.float32, device=x.device)
    _ok(lmhead_quantize_fp8(rows, cols, block_rows, x, q, scale), "lmhead_quantize_fp8")
    return q, scale


@_on_device_of(0)
def logits_fp8(a, a_scale, w, w_scale, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None):
    """Logits [n, vocab] of 8-bit rows (quantize_fp8 with block_rows 1, or
    rms_norm_quant) and an 8-bit W (block_rows 128). out: a [n, vocab] tensor
    to write, rows contiguous, any row stride; its dtype is then the output's."""
    e4m3 = (torch.float8_e4m3fn,)
    _check_gpu("a", a, e4m3, (None, None))
    _check_gpu("w", w, e4m3, (None, a.shape[1]), a.device)
    n, hidden = a.shape
    vocab = w.shape[0]
    if hidden % FP8_BLOCK != 0:
        raise LMHeadError(LMHEAD_ERR_SHAPE, "lmhead_logits_fp8")
    f32 = (torch.float32,)
    _check_gpu("a_scale", a_scale, f32, (n, hidden // FP8_BLOCK), a.device)
    _check_gpu("w_scale", w_scale, f32, (-(-vocab // FP8_BLOCK), hidden // FP8_BLOCK), a.device)
    if out is None:
        if out_dtype not in _DTYPES:
            raise ValueError("out_dtype must be bfloat16 or float32")
        out = torch.empty(n, vocab, dtype=out_dtype, device=a.device)
    ld = _row_stride("out", out, (n, vocab), a.device)
    p = lmhead_fp8_problem(n, vocab, hidden, ld, _DTYPES[out.dtype], 0)
    ws = _workspace(ws, lmhead_logits_fp8_workspace_size(p), a.device, lmhead_logits_fp8, p, 6)
    _ok(lmhead_logits_fp8(p, a, a_scale, w, w_scale, out, ws, ws.numel()), "lmhead_logits_fp8")
    return out


def _row_stride(name, t, shape, device) -> int:
    """Row stride of a [n, vocab] bf16 / fp32 tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on a GPU device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on the inputs' device")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float32")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be [n, vocab]")
    n, vocab = t.shape
    if vocab > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    if n <= 1:
        return vocab
    if t.stride(0) < vocab:
        raise ValueError(f"{name}'s rows must not overlap")
    return t.stride(0)


@_on_device_of(0)
def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, want_logprob: bool = True,
           ws: Optional[torch.Tensor] = None):
    """One token per row: (token int32 [n], logprob fp32 [n] or None); see
    lmhead_sample for the rule. logits: bf16 or fp32 [n, vocab], rows contiguous.
    Each filter is a number for all rows, a device tensor [n] (fp32; top_k
    int32) or None (off). Bad rows give token -1 (logprob NaN), rows with every
    token masked token -1 (logprob 0); pass ws to read the error word."""
    ld = _row_stride("logits", logits, None, None)
    n, vocab = logits.shape
    dev = logits.device
    _check_f32("u", u, (n,), dev, required=n > 0)
    rows = {}
    scalars = {}
    for name, v in (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)):
        if isinstance(v, torch.Tensor):
            _check_gpu(name, v, (torch.int32 if name == "top_k" else torch.float32,), (n,), dev)
            rows[name] = v
        elif v is not None:
            # as the fp32 number that the C call gets, where 0 means off
            if name in ("temperature", "top_p") and not ctypes.c_float(v).value > 0:
                raise ValueError(f"{name} must be positive")
            if name == "top_k" and (v != int(v) or not -1 << 31 <= v < 1 << 31):
                raise ValueError("top_k must be a 32-bit integer")
            scalars[name] = v
    p = lmhead_sample_problem(n, vocab, ld, _DTYPES[logits.dtype], int(scalars.get("top_k", 0)),
                              float(scalars.get("temperature", 0.0)), float(scalars.get("top_p", 0.0)),
                              float(scalars.get("min_p", 0.0)), 0, _p(rows.get("temperature")),
                              _p(rows.get("top_k")), _p(rows.get("top_p")), _p(rows.get("min_p")))
    ws = _workspace(ws, lmhead_sample_workspace_size(p), dev, lmhead_sample, p, 5)
    token = torch.empty(n, dtype=torch.int32, device=dev)
    logprob = torch.empty(n, dtype=torch.float32, device=dev) if want_logprob else None
    _ok(lmhead_sample(p, logits, u, token, logprob, ws, ws.numel()), "lmhead_sample")
    return token, logprob


def next_token(x, norm_weight, w, w_scale, u, residual=None, eps: float = 1e-6, weight_offset: float = 0.0,
               temperature=None, top_k=None, top_p=None, min_p=None, logits_dtype=torch.float32):
    """The answer path in one call: final norm of the last hidden states x (+
    residual) in 8 bits, logits against an 8-bit W, one sampled token per row.
    Returns (token, logprob, residual_out or None)."""
    q, scale, r = rms_norm_quant(x, norm_weight, residual, eps, weight_offset)
    logits = logits_fp8(q, scale, w, w_scale, out_dtype=logits_dtype)
    token, logprob = sample(logits, u, temperature, top_k, top_p, min_p)
    return token, logprob, r
