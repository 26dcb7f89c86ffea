"""Embedding with the LM head's weight (argument marshalling only; the arithmetic
runs in the CUDA library, see flce_embedding_* in include/flce.h).

  embedding_forward(weight, ids, scale=1.0, ignore_index=-100) -> [..., H]
  embedding_backward(d_out, ids, vocab, scale=1.0, ...) -> d_weight [V, H], written
      whole or added into a given buffer (tied weights: the LM head's gradient)
  fused_embedding(...)  the differentiable form
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _native
from .flce import _DTYPES, _lib, _ptr, _stream, check_workspace, on_device, status


_ID_DTYPES = (torch.int64, torch.int32, torch.int16, torch.uint8, torch.int8)


def _ids(ids: torch.Tensor, device) -> torch.Tensor:
    if ids.device != device:
        raise ValueError("ids must be a CUDA tensor on the weight's device")
    if ids.dtype not in _ID_DTYPES:
        raise TypeError("ids must be integers")
    y = ids if ids.dim() == 1 else ids.reshape(-1)
    return y.to(torch.int64).contiguous() if y.dtype != torch.int64 else y.contiguous()


def embedding_forward(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
                      ignore_index: int = -100, check_status: bool = False) -> torch.Tensor:
    """scale * weight[ids] [..., H] in the weight's dtype (bfloat16 or float32), rounded
    once; zeros where ids is ignore_index (or outside [0, V), which check_status
    raises for)."""
    if not weight.is_cuda:
        raise ValueError("weight must be a CUDA tensor")
    if weight.dtype not in _DTYPES:
        raise TypeError("weight must be bfloat16 or float32")
    if weight.dim() != 2:
        raise ValueError("weight must be [vocab, hidden]")
    dev = weight.device
    y = _ids(ids, dev)
    w = weight.contiguous()
    V, H = w.shape
    out = torch.empty(ids.shape + (H,), dtype=w.dtype, device=dev)
    word = torch.empty(1, dtype=torch.int32, device=dev) if check_status else None
    with on_device(dev):
        st = _lib().flce_embedding_forward(_ptr(w), _ptr(y), y.shape[0], H, V, int(ignore_index),
                                           float(scale), _DTYPES[w.dtype], _ptr(out), _ptr(word),
                                           _stream(dev))
    _native.check(st, "flce_embedding_forward")
    if check_status and int(word) != 0:
        raise _native.FlceError(_native.LABEL_RANGE, "flce_embedding_forward (device status)")
    return out


def embedding_workspace_bytes(N: int, H: int, V: int) -> int:
    """Workspace of embedding_backward (0 for invalid sizes)."""
    return int(_lib().flce_embedding_workspace_bytes(N, H, V))


def embedding_backward(d_out: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0,
                       ignore_index: int = -100, padding_idx: Optional[int] = None,
                       d_weight: Optional[torch.Tensor] = None, accumulate: bool = False,
                       grad_dtype: torch.dtype = torch.float32,
                       workspace: Optional[torch.Tensor] = None,
                       check_status: bool = False) -> torch.Tensor:
    """dWeight [vocab, H] of embedding_forward for the upstream gradient d_out
    [..., H] (bfloat16 or float32), float32 or bfloat16 (a given d_weight's dtype, else
    grad_dtype): summed in fp32, rounded once.  accumulate: added into the given d_weight, of
    which only the rows that ids name are read and written; else every row is
    written.  padding_idx: an id whose row gets no gradient."""
    if not d_out.is_cuda:
        raise ValueError("d_out must be a CUDA tensor")
    if d_out.dtype not in _DTYPES:
        raise TypeError("d_out must be bfloat16 or float32")
    dev = d_out.device
    y = _ids(ids, dev)
    if d_out.dim() < 1 or tuple(d_out.shape[:-1]) != tuple(ids.shape):
        raise ValueError("d_out must be [*ids.shape, hidden]")
    N, H, V = y.shape[0], d_out.shape[-1], int(vocab)
    if padding_idx is not None and not 0 <= padding_idx < V:
        raise ValueError("padding_idx must lie in [0, vocab)")
    if accumulate and d_weight is None:
        raise ValueError("accumulating needs an existing d_weight")
    if d_weight is None:
        if grad_dtype not in _DTYPES:
            raise TypeError("grad_dtype must be float32 or bfloat16")
        if V < 1:
            raise ValueError("vocab must be positive")
        d_weight = torch.empty((V, H), dtype=grad_dtype, device=dev)
    elif (tuple(d_weight.shape) != (V, H) or d_weight.dtype not in _DTYPES
          or not d_weight.is_contiguous() or d_weight.device != dev):
        raise ValueError(f"d_weight must be a contiguous float32 or bfloat16 {[V, H]} tensor "
                         f"on {dev}")
    g = d_out.reshape(N, H).contiguous()
    flags = ((_native.ACCUMULATE_DWEIGHT if accumulate else 0)
             | (_native.DWEIGHT_BF16 if d_weight.dtype == torch.bfloat16 else 0))
    if workspace is None:
        n = embedding_workspace_bytes(N, H, V)
        if n == 0:
            raise ValueError("invalid sizes")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        check_workspace(workspace, dev)
    with on_device(dev):
        st = _lib().flce_embedding_backward(
            _ptr(g), _ptr(y), N, H, V, int(ignore_index),
            -1 if padding_idx is None else int(padding_idx), float(scale), _DTYPES[g.dtype],
            _ptr(d_weight), flags, _ptr(workspace), workspace.numel(), _stream(dev))
    _native.check(st, "flce_embedding_backward")
    if check_status:
        _native.check(status(workspace), "flce_embedding_backward (device status)")
    return d_weight


class _EmbeddingFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, ignore_index, padding_idx):
        ctx.save_for_backward(ids)
        ctx.cfg = (scale, ignore_index, padding_idx, weight.shape[0], weight.dtype)
        return embedding_forward(weight, ids, scale, ignore_index)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        if not ctx.needs_input_grad[0]:
            return (None,) * 5
        ids, = ctx.saved_tensors
        scale, ignore_index, padding_idx, vocab, dtype = ctx.cfg
        # in the parameter's own dtype (bf16 rounded once from fp32)
        return (embedding_backward(d_out, ids, vocab, scale, ignore_index, padding_idx,
                                   grad_dtype=dtype),) + (None,) * 4


def fused_embedding(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
                    ignore_index: int = -100, padding_idx: Optional[int] = None) -> torch.Tensor:
    """Differentiable embedding_forward; padding_idx as F.embedding's (looked up, but
    without a gradient)."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise ValueError("padding_idx must lie in [0, vocab)")
    return _EmbeddingFunction.apply(weight, ids, scale, ignore_index, padding_idx)
