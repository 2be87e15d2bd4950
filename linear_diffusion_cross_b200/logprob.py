"""Log-probabilities of given tokens, entropy and the best alternatives from
hidden states and the head's weight, without the logits in memory (the
workspace holds candidates of every slice of the vocabulary instead: 0.08 GB
for 4096 tokens of 151936 entries, 0.7 GB with 8 alternatives, at most about
1.1 GB for any number of tokens).

``fused_linear_logprobs(x, token, weight, ...)`` is what scoring, decoding and
policy-gradient training ask of the head that ``FusedLinearDiffusionCrossEntropyLoss``
trains.  ``logprob`` and ``entropy`` are differentiable in x, weight and bias;
the backward recomputes the logits in one sweep (``fldce_logprob_bwd``).  The
weight may be a ``W4Weight`` (forward only).

Workspaces come from PyTorch's allocator per call, on the call's own stream:
calls on several streams, and captured graphs, share none.
"""
from __future__ import annotations

import functools
from typing import NamedTuple, Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .module import _dtype_code, refuse_forward_mode
from .w4 import W4Weight, check_w4_input, dense, on_device_of, raw_stream

_MAX_N = (1 << 31) - 1
_INTS = frozenset((torch.int64, torch.int32, torch.int16, torch.int8, torch.uint8))


class _Plan:
    """A plan's host state (no device memory), freed with the last reference."""

    __slots__ = ("handle", "lse_pair", "_sizes")

    def __init__(self, dtype: torch.dtype, D: int, V: int, logit_scale: float, ignore_index: int,
                 chunk_n: int):
        self.handle = None
        self._sizes = {}
        # fp32 gradients would show the rounding of lse
        self.lse_pair = dtype == torch.float32
        self.handle, _ = B.fldce_create(_dtype_code(dtype), D, V, _MAX_N, chunk_N=chunk_n,
                                        logit_scale=logit_scale, ignore_index=ignore_index,
                                        flags=B.FLDCE_FLAG_LSE_PAIR if self.lse_pair else 0)

    def __del__(self):
        if self.handle is not None:
            try:
                B.fldce_destroy(self.handle)
            except Exception:      # the interpreter is going down
                pass

    def _size(self, key: tuple, f, *args) -> int:
        n = self._sizes.get(key)
        if n is None:
            if len(self._sizes) >= 1024:
                self._sizes.clear()
            n = self._sizes[key] = f(self.handle, *args)
        return n

    def workspace_size(self, N: int, top_k: int) -> int:
        return self._size((N, top_k), B.fldce_logprob_workspace_size, N, top_k)

    def bwd_workspace_size(self, N: int) -> int:
        return self._size((N,), B.fldce_logprob_bwd_workspace_size, N)


# The latest configurations' plans.  One that drops out lives on in the calls
# and autograd graphs that hold it; a logit_scale that changes each step leaves
# nothing behind.
_plan = functools.lru_cache(maxsize=64)(_Plan)


class LinearLogProbs(NamedTuple):
    """Results of ``fused_linear_logprobs``; leading dimensions are x's."""

    logprob: Optional[torch.Tensor]        # fp32 [...]: log p(token), 0 where ignored
    entropy: torch.Tensor                  # fp32 [...]
    lse: torch.Tensor                      # fp32 [...]
    top_ids: Optional[torch.Tensor]        # int32 [..., top_k], best first
    top_logprobs: Optional[torch.Tensor]   # fp32 [..., top_k]


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    # (an empty tensor may have no address)
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _forward(x, weight, bias, token, plan, top_k):
    """The five results, and the lse that the backward wants (with what rounding
    took off it behind it, in fp32)."""
    N = x.shape[0]
    dev = x.device
    f32 = torch.float32
    with on_device_of(x):
        logprob = None if token is None else torch.empty(N, dtype=f32, device=dev)
        entropy = torch.empty(N, dtype=f32, device=dev)
        lse_all = torch.empty(2 * N if plan.lse_pair else N, dtype=f32, device=dev)
        lse = lse_all[:N] if plan.lse_pair else lse_all
        ids = top = None
        if top_k:
            ids = torch.empty((N, top_k), dtype=torch.int32, device=dev)
            top = torch.empty((N, top_k), dtype=f32, device=dev)
        if N == 0:
            return logprob, entropy, lse, ids, top, lse_all
        nbytes = plan.workspace_size(N, top_k)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if isinstance(weight, W4Weight):
            w, w4, scales, group = None, weight.packed.data_ptr(), weight.scales.data_ptr(), \
                weight.group_size
        else:
            w, w4, scales, group = weight.data_ptr(), None, None, 0
        B.fldce_logprob(plan.handle, B.fldce_logprob_call(
            x.data_ptr(), w, w4, scales, _ptr(bias), _ptr(token), N, group, top_k, _ptr(logprob),
            entropy.data_ptr(), lse.data_ptr(), _ptr(ids), _ptr(top), ws.data_ptr(), nbytes, None,
            raw_stream(dev)))
    return logprob, entropy, lse, ids, top, lse_all


class FusedLinearLogProbsFunction(torch.autograd.Function):
    """log p and entropy with gradients; lse and the alternatives without."""

    @staticmethod
    def forward(ctx, x, weight, bias, token, plan, top_k):
        logprob, entropy, lse, ids, top, lse_all = _forward(x, weight, bias, token, plan, top_k)
        ctx.set_materialize_grads(False)
        ctx.plan = plan
        ctx.save_for_backward(x, weight, bias, token, lse_all, entropy)
        ctx.mark_non_differentiable(*(t for t in (lse, ids, top) if t is not None))
        return logprob, entropy, lse, ids, top

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogprob, dentropy, *_):
        x, weight, bias, token, lse, entropy = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        if dlogprob is None and dentropy is None:
            return None, None, None, None, None, None
        if dlogprob is not None:
            dlogprob = dlogprob.float().contiguous()
        if dentropy is not None:
            dentropy = dentropy.float().contiguous()
        N = x.shape[0]
        dev = x.device
        with on_device_of(x):
            dH = torch.empty_like(x) if need_x else None
            dW = torch.empty_like(weight) if need_w else None
            db = torch.empty_like(bias) if need_b else None
            nbytes = ctx.plan.bwd_workspace_size(N)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            B.fldce_logprob_bwd(ctx.plan.handle, B.fldce_logprob_grad_call(
                _ptr(x), weight.data_ptr(), _ptr(bias), _ptr(token), N, _ptr(lse), _ptr(entropy),
                _ptr(dlogprob), _ptr(dentropy), _ptr(dH), _ptr(dW), _ptr(db), ws.data_ptr(),
                nbytes, None, raw_stream(dev)))
        return dH, dW, db, None, None, None


def fused_linear_logprobs(x: torch.Tensor, token: Optional[torch.Tensor],
                          weight: Union[torch.Tensor, W4Weight],
                          bias: Optional[torch.Tensor] = None, *, top_k: int = 0,
                          logit_scale: float = 1.0, ignore_index: int = -100,
                          chunk_n: int = 0) -> LinearLogProbs:
    """x [..., D], token [...] int64 (or None), weight [V, D] or ``W4Weight``,
    bias [V] or None -> ``LinearLogProbs``.

    z = logit_scale * (x W^T + bias).  A token equal to ``ignore_index``, or
    outside [0, V), has logprob 0 and no gradient through it.  ``top_ids`` are
    ordered by the exact logits, equal ones by lowest id, among at least
    ``top_k + 3`` entries that have the largest fp32 logits (so they are the
    exact best unless more than three others come within the fp32 error of the
    last); a bias of -inf takes an entry out.  ``chunk_n`` (0: the library's
    choice) bounds the tokens whose logit gradient the backward holds at a time.
    Forward-mode derivatives are refused.
    """
    w4 = isinstance(weight, W4Weight)
    if w4:
        check_w4_input(x, weight, bias)
    elif weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and weight {tuple(weight.shape)} do not match")
    elif x.dtype != weight.dtype:
        raise TypeError("x and weight must have the same dtype")
    V, D = weight.shape
    if bias is not None and (bias.shape != (V,) or bias.dtype != x.dtype):
        raise ValueError(f"bias {tuple(bias.shape)} {bias.dtype} does not match weight")
    if token is not None and token.shape != x.shape[:-1]:
        raise ValueError(f"x={tuple(x.shape)}, token={tuple(token.shape)}")
    if token is not None and token.dtype not in _INTS:
        raise TypeError(f"token has to hold integers, got {token.dtype}")
    if not 0 <= top_k <= min(B.FLDCE_MAX_TOP_K, V):
        raise ValueError(f"top_k {top_k} is not in 0..{min(B.FLDCE_MAX_TOP_K, V)}")
    _dtype_code(x.dtype)
    if not w4:
        refuse_forward_mode(x, weight, bias)
    if not x.is_cuda:
        raise RuntimeError("the fused log-probabilities run on CUDA tensors only")
    dev = x.device
    if weight.device != dev or (bias is not None and bias.device != dev) or (
            token is not None and token.device != dev):
        raise ValueError("x, token, weight and bias are on different devices")
    lead = x.shape[:-1]
    x2 = dense(x if len(lead) == 1 else x.reshape(-1, D))
    if not w4:
        weight = dense(weight)
    bias = dense(bias)
    if token is not None:
        if len(lead) != 1:
            token = token.reshape(-1)
        if token.dtype != torch.int64 or not token.is_contiguous():
            token = token.to(torch.int64).contiguous()
    plan = _plan(x.dtype, D, V, float(logit_scale), int(ignore_index), int(chunk_n))
    if torch.is_grad_enabled() and not w4 and (
            x2.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)):
        out = FusedLinearLogProbsFunction.apply(x2, weight, bias, token, plan, top_k)
    else:
        out = _forward(x2, weight, bias, token, plan, top_k)[:5]
    if len(lead) != 1:
        out = (*(None if t is None else t.view(lead) for t in out[:3]),
               *(None if t is None else t.view(*lead, top_k) for t in out[3:]))
    return LinearLogProbs(*out)


class FusedLinearLogProbs(torch.nn.Module):
    """``fused_linear_logprobs`` with its options held by a module."""

    def __init__(self, top_k: int = 0, logit_scale: float = 1.0, ignore_index: int = -100,
                 chunk_n: int = 0):
        super().__init__()
        if not 0 <= top_k <= B.FLDCE_MAX_TOP_K:
            raise ValueError(f"top_k {top_k} is not in 0..{B.FLDCE_MAX_TOP_K}")
        self.top_k = top_k
        self.logit_scale = logit_scale
        self.ignore_index = ignore_index
        self.chunk_n = chunk_n

    def forward(self, x: torch.Tensor, token: Optional[torch.Tensor],
                weight: Union[torch.Tensor, W4Weight],
                bias: Optional[torch.Tensor] = None) -> LinearLogProbs:
        return fused_linear_logprobs(x, token, weight, bias, top_k=self.top_k,
                                     logit_scale=self.logit_scale,
                                     ignore_index=self.ignore_index, chunk_n=self.chunk_n)
