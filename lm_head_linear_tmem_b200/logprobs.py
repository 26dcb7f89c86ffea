"""Scoring with the LM head: log probabilities of given tokens, entropy and top
alternatives of softmax(softcap(hidden . weight^T) / temperature), without the
[tokens, vocab] logits (argument marshalling only; the arithmetic runs in the
CUDA library, see flce_logprobs_forward_ex in include/flce.h).

  logprobs_forward(hidden, weight, tokens=None, ignore_index=-100, softcap=0.0,
                   temperature=1.0, top_k=0)
      -> Logprobs(logprobs, entropy, lse, top_logprobs, top_ids, saved)
  logprobs_backward(hidden, weight, tokens, saved, d_logprobs, d_entropy)
      -> (d_hidden, d_weight)
  fused_linear_logprobs(...)  the differentiable form: gradients of the log
      probabilities and the entropy flow to hidden and weight
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _native
from .flce import (_DTYPES, _lib, _prep, _ptr, _stream, alloc_grads, alloc_workspace, check_workspace,
                   on_device, status)


class Logprobs(NamedTuple):
    logprobs: Optional[torch.Tensor]      # float32 [...]; None without tokens
    entropy: torch.Tensor                 # float32 [...]
    lse: torch.Tensor                     # float32 [...]
    top_logprobs: Optional[torch.Tensor]  # float32 [..., top_k]; None with top_k=0
    top_ids: Optional[torch.Tensor]       # int64 [..., top_k]
    saved: torch.Tensor                   # float32 [3, N]: logprobs_backward's


def logprobs_workspace_bytes(N: int, H: int, V: int, dtype: torch.dtype = torch.bfloat16,
                             top_k: int = 0) -> int:
    """Workspace of logprobs_forward (0 for invalid sizes)."""
    return int(_lib().flce_logprobs_workspace_bytes(N, H, V, _DTYPES[dtype], int(top_k)))


def logprobs_forward(hidden: torch.Tensor, weight: torch.Tensor,
                     tokens: Optional[torch.Tensor] = None, ignore_index: int = -100,
                     softcap: float = 0.0, temperature: float = 1.0, top_k: int = 0,
                     workspace: Optional[torch.Tensor] = None,
                     check_status: bool = False, *, _own_storage: bool = False) -> Logprobs:
    """Scores hidden [..., H] with the LM head weight [V, H] (bfloat16 or float32).

    tokens [...]: the given tokens; rows whose token is ignore_index take no part
    (outputs 0, ids -1).  Without tokens every row is scored and `logprobs` is
    None.  top_k (at most 32): that many alternatives per row, best first, the
    lowest id of equal logits first."""
    lead = hidden.shape[:-1]
    h2, w, y = _prep(hidden, weight, tokens)
    N, H = h2.shape
    V = w.shape[0]
    dev = h2.device
    k = int(top_k)
    if not 0 <= k <= min(V, _native.MAX_TOP_K):
        raise ValueError(f"top_k must lie in [0, {min(V, _native.MAX_TOP_K)}]")
    if workspace is None:
        n = logprobs_workspace_bytes(N, H, V, h2.dtype, k)
        if n == 0:
            raise ValueError("invalid sizes")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    else:
        check_workspace(workspace, dev)
    if _own_storage:  # an autograd function's outputs, which a caller may change in place
        saved = torch.empty((3, N), dtype=torch.float32, device=dev)
        entropy, lse = (torch.empty(lead, dtype=torch.float32, device=dev) for _ in range(2))
        logprobs = None if y is None else torch.empty_like(lse)
    else:  # one allocation
        f = torch.empty((5 if y is None else 6, *lead), dtype=torch.float32, device=dev)
        entropy, lse, *rest = f[3:].unbind(0)
        saved, logprobs = f[:3].view(3, N), rest[0] if rest else None
    top_lp = torch.empty((*lead, k), dtype=torch.float32, device=dev) if k else None
    top_ids = torch.empty((*lead, k), dtype=torch.int64, device=dev) if k else None
    with on_device(dev):
        st = _lib().flce_logprobs_forward_ex(
            _ptr(h2), _ptr(w), _ptr(y), N, H, V, int(ignore_index), float(softcap),
            float(temperature), k, _DTYPES[h2.dtype], _ptr(logprobs), _ptr(entropy), _ptr(lse),
            _ptr(saved), _ptr(top_lp), _ptr(top_ids), _ptr(workspace), workspace.numel(),
            _stream(dev))
    _native.check(st, "flce_logprobs_forward")
    if check_status:
        _native.check(status(workspace), "flce_logprobs_forward (device status)")
    return Logprobs(logprobs, entropy, lse, top_lp, top_ids, saved)


def _row_grad(t: Optional[torch.Tensor], name: str, N: int, dev) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.numel() != N or t.device != dev:
        raise ValueError(f"{name} must have one entry per token, on {dev}")
    return t.reshape(-1).to(torch.float32).contiguous()


def logprobs_backward(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor,
                      saved: torch.Tensor, d_logprobs: Optional[torch.Tensor] = None,
                      d_entropy: Optional[torch.Tensor] = None, ignore_index: int = -100,
                      softcap: float = 0.0, temperature: float = 1.0,
                      workspace: Optional[torch.Tensor] = None,
                      d_hidden: Optional[torch.Tensor] = None,
                      d_weight: Optional[torch.Tensor] = None,
                      accumulate_d_hidden: bool = False, accumulate_d_weight: bool = False,
                      grad_dtype: torch.dtype = torch.float32,
                      compute_d_hidden: bool = True, compute_d_weight: bool = True,
                      check_status: bool = False
                      ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """dHidden [N, H] and dWeight [V, H] of sum(d_logprobs * logprobs + d_entropy *
    entropy), either of them None for zeros.  `saved` is logprobs_forward's; the gradient buffers and switches as for `backward`."""
    if tokens is None:
        raise ValueError("the backward needs tokens (any valid ones if only d_entropy is given)")
    h2, w, y = _prep(hidden, weight, tokens)
    N, H = h2.shape
    V = w.shape[0]
    dev = h2.device
    a = _row_grad(d_logprobs, "d_logprobs", N, dev)
    b = _row_grad(d_entropy, "d_entropy", N, dev)
    if tuple(saved.shape) != (3, N) or saved.dtype != torch.float32 or saved.device != dev:
        raise ValueError(f"saved must be logprobs_forward's float32 [3, {N}] tensor on {dev}")
    saved = saved.contiguous()
    d_hidden, d_weight, flags = alloc_grads(N, H, V, dev, d_hidden, d_weight, accumulate_d_hidden,
                                            accumulate_d_weight, grad_dtype, compute_d_hidden,
                                            compute_d_weight)
    if workspace is None:
        workspace = alloc_workspace(N, H, V, h2.dtype, dev, flags)
    else:
        check_workspace(workspace, dev)
    with on_device(dev):
        st = _lib().flce_logprobs_backward_ex(
            _ptr(h2), _ptr(w), _ptr(y), _ptr(saved), N, H, V, int(ignore_index),
            float(softcap), float(temperature), _DTYPES[h2.dtype], _ptr(a), _ptr(b),
            _ptr(d_hidden), _ptr(d_weight), flags, _ptr(workspace), workspace.numel(),
            _stream(dev))
    _native.check(st, "flce_logprobs_backward")
    if check_status:
        _native.check(status(workspace), "flce_logprobs_backward (device status)")
    return d_hidden, d_weight


class _LogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, tokens, ignore_index, softcap, temperature, top_k):
        out = logprobs_forward(hidden, weight, tokens, ignore_index, softcap, temperature, top_k,
                               _own_storage=True)
        ctx.save_for_backward(hidden, weight, tokens, out.saved)
        ctx.cfg = (ignore_index, softcap, temperature)
        ctx.mark_non_differentiable(*(t for t in out[2:] if t is not None))
        ctx.set_materialize_grads(False)
        return tuple(out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_logprobs, d_entropy, *_):
        hidden, weight, tokens, saved = ctx.saved_tensors
        ignore_index, softcap, temperature = ctx.cfg
        need_dh, need_dw = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_dh or need_dw) or (d_logprobs is None and d_entropy is None):
            return (None,) * 7
        if tokens is None:  # only the entropy's gradient: any valid token will do
            tokens = torch.zeros(saved.shape[1], dtype=torch.int64, device=saved.device)
            ignore_index = -100
        # gradients in the parameters' own dtype (bf16 rounded once from fp32)
        dh = (torch.empty(hidden.shape, dtype=hidden.dtype, device=hidden.device)
              .view(-1, hidden.shape[-1]) if need_dh else None)
        dw = torch.empty(weight.shape, dtype=weight.dtype, device=weight.device) \
            if need_dw else None
        logprobs_backward(hidden, weight, tokens, saved, d_logprobs, d_entropy, ignore_index,
                          softcap, temperature, d_hidden=dh, d_weight=dw,
                          compute_d_hidden=need_dh, compute_d_weight=need_dw)
        return ((dh.view(hidden.shape) if need_dh else None), dw) + (None,) * 5


def fused_linear_logprobs(hidden: torch.Tensor, weight: torch.Tensor,
                          tokens: Optional[torch.Tensor] = None, ignore_index: int = -100,
                          softcap: float = 0.0, temperature: float = 1.0,
                          top_k: int = 0) -> Logprobs:
    """Differentiable logprobs_forward: gradients of `logprobs` and `entropy` flow
    to hidden and weight (policy-gradient losses, entropy bonuses); the other outputs
    carry none."""
    return Logprobs(*_LogprobsFunction.apply(hidden, weight, tokens, ignore_index, softcap,
                                             temperature, top_k))
