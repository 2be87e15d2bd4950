"""A head weight in 4 bits: ``W4Weight``, ``quantize_w4`` and ``linear_w4``.

``W[v, d] = q[v, d] * scale[v, d // group_size]`` with ``q`` a two's
complement nibble: byte i of a row of ``packed`` holds element 2i in its low
half and element 2i + 1 in its high half, ``scales`` holds one bf16 number for
each run of ``group_size`` elements of a row.  For a few tokens at a time a
head is bound by the bytes of its weight, of which 4 bits leave about a
quarter.  ``fused_linear_logprobs`` takes a ``W4Weight`` in place of a tensor.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import torch

from . import binding as B
from .module import _dtype_code, refuse_forward_mode

GROUP_SIZES = (32, 64, 128)


def dense(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """``t`` contiguous from a 16-byte boundary on, as the library takes it."""
    if t is None:
        return None
    if not t.is_contiguous():
        t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def raw_stream(device: torch.device) -> int:
    """The handle of the device's current stream (for a call a token, without
    the Stream object that torch.cuda.current_stream makes)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


class on_device_of:
    """Make the device of ``t`` the current one (the library works on that)."""

    def __init__(self, t: torch.Tensor):
        self.to = t.device.index
        self.back = None

    def __enter__(self):
        cur = torch.cuda.current_device()
        if cur != self.to:
            torch.cuda.set_device(self.to)
            self.back = cur

    def __exit__(self, *exc):
        if self.back is not None:
            torch.cuda.set_device(self.back)


@dataclasses.dataclass(frozen=True, eq=False)
class W4Weight:
    """A [V, D] weight in 4 bits: ``packed`` uint8 [V, D/2], ``scales`` bf16 [V, ceil(D/group_size)].
    Two are equal if they are the same object, as parameters are."""

    packed: torch.Tensor
    scales: torch.Tensor
    group_size: int

    def __post_init__(self):
        p, s, g = self.packed, self.scales, self.group_size
        if g not in GROUP_SIZES:
            raise ValueError(f"group_size {g} is not one of {GROUP_SIZES}")
        if p.dim() != 2 or p.dtype != torch.uint8:
            raise TypeError(f"packed has to be a uint8 matrix, got {p.dtype} {tuple(p.shape)}")
        V, D = p.shape
        D *= 2
        if V == 0 or D == 0 or D % 32:
            raise ValueError(f"a 4-bit weight needs D a multiple of 32 and V > 0, got {(V, D)}")
        if s.dtype != torch.bfloat16 or s.shape != (V, -(-D // g)):
            raise ValueError(f"scales have to be bfloat16 {(V, -(-D // g))}, got {s.dtype} "
                             f"{tuple(s.shape)}")
        if p.device != s.device:
            raise ValueError("packed and scales are on different devices")
        for name, t in (("packed", p), ("scales", s)):
            d = dense(t)
            if d is not t:
                object.__setattr__(self, name, d)

    @property
    def shape(self) -> tuple:
        V, half = self.packed.shape
        return V, 2 * half

    @property
    def device(self) -> torch.device:
        return self.packed.device


def quantize_w4(weight: torch.Tensor, group_size: int = 128) -> W4Weight:
    """Round a bf16 or fp32 ``weight`` [V, D] to 4 bits: per group of a row,
    scale = bf16(max|w| / 7) and q = round(w / scale) in [-7, 7].  The weights
    have to be finite."""
    if weight.dim() != 2:
        raise ValueError(f"weight has to be a matrix, got {tuple(weight.shape)}")
    if group_size not in GROUP_SIZES:
        raise ValueError(f"group_size {group_size} is not one of {GROUP_SIZES}")
    code = _dtype_code(weight.dtype)
    V, D = weight.shape
    if V == 0 or D == 0 or D % 32:
        raise ValueError(f"a 4-bit weight needs D a multiple of 32 and V > 0, got {(V, D)}")
    if not weight.is_cuda:
        raise RuntimeError("quantize_w4 runs on CUDA tensors only")
    weight = dense(weight.detach())
    with on_device_of(weight):
        packed = torch.empty(V, D // 2, dtype=torch.uint8, device=weight.device)
        scales = torch.empty(V, -(-D // group_size), dtype=torch.bfloat16, device=weight.device)
        B.fldce_w4_quantize(weight, code, V, D, group_size, packed, scales,
                            torch.cuda.current_stream(weight.device))
    return W4Weight(packed, scales, group_size)


def check_w4_input(x: torch.Tensor, weight: W4Weight, bias: Optional[torch.Tensor]):
    V, D = weight.shape
    if x.dim() < 1 or x.shape[-1] != D:
        raise ValueError(f"x {tuple(x.shape)} and weight {tuple(weight.shape)} do not match")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"a 4-bit weight takes bfloat16 inputs, got {x.dtype}")
    if bias is not None and (bias.shape != (V,) or bias.dtype != x.dtype):
        raise ValueError(f"bias {tuple(bias.shape)} {bias.dtype} does not match weight")
    if torch.is_grad_enabled() and (x.requires_grad or weight.scales.requires_grad or
                                    (bias is not None and bias.requires_grad)):
        raise RuntimeError("a 4-bit weight has no gradient path: call it under torch.no_grad()")
    refuse_forward_mode(x, weight.scales, bias)


def linear_w4(x: torch.Tensor, weight: W4Weight, bias: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Logits ``x @ W.T + bias`` [..., V] of a few tokens ``x`` [..., D] (bf16),
    summed in fp32 and rounded once to ``out_dtype`` (float32 or bfloat16)."""
    check_w4_input(x, weight, bias)
    code = _dtype_code(out_dtype)
    if not x.is_cuda:
        raise RuntimeError("linear_w4 runs on CUDA tensors only")
    if weight.device != x.device or (bias is not None and bias.device != x.device):
        raise ValueError("x, weight and bias are on different devices")
    V, D = weight.shape
    x2 = dense(x if x.dim() == 2 else x.reshape(-1, D))
    bias = dense(bias)
    with on_device_of(x2):
        out = torch.empty((x2.shape[0], V), dtype=out_dtype, device=x.device)
        B.fldce_w4_linear(x2, x2.shape[0], weight.packed, weight.scales, weight.group_size, bias,
                          V, D, out, code, stream=raw_stream(x.device))
    return out if x.dim() == 2 else out.view(*x.shape[:-1], V)
