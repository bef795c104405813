"""Weights in the 4-bit layouts that ep_matvec_w4 reads.

``quantize_w4`` lays a weight tensor out once, when a model is loaded: codes two to a
byte (the even column in the low four bits), one scale to a group of consecutive columns.
It works on the tensor's own device and needs no library."""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import EP_W4_E2M1, EP_W4_INT

E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of codes 0..7; codes 8..15 negative


@dataclass
class W4Weights:
    """Codes [..., N, K/2] bytes; scales [..., N, K/group_size] (bf16, or for EP_W4_E2M1
    exponent bytes); zeros the same shape in bytes, or None (8 everywhere)."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: torch.Tensor | None
    w_format: int
    group_size: int

    def to(self, device) -> "W4Weights":
        return W4Weights(self.codes.to(device), self.scales.to(device),
                         None if self.zeros is None else self.zeros.to(device),
                         self.w_format, self.group_size)


def quantize_w4(w: torch.Tensor, w_format: int = EP_W4_INT, group_size: int = 32,
                zeros: bool = True) -> W4Weights:
    """The nearest codes for ``w`` [..., K], whatever its strides; the results are contiguous.
    EP_W4_INT: a group's scale is its range over 15 with a zero point each (``zeros``), or its
    largest magnitude over 7 around code 8; EP_W4_E2M1: the smallest power of two at which no
    code saturates."""
    K = w.shape[-1]
    if w_format not in (EP_W4_INT, EP_W4_E2M1):
        raise ValueError(f"w_format {w_format}")
    if group_size not in ((32,) if w_format == EP_W4_E2M1 else (32, 64, 128)) or K % group_size:
        raise ValueError(f"group_size {group_size} for K = {K}")
    # (contiguous: elementwise results keep their input's strides, and the kernels go by address)
    g = w.contiguous().float().unflatten(-1, (K // group_size, group_size))
    zero = None
    if w_format == EP_W4_E2M1:
        top = g.abs().amax(-1)
        # frexp: top / 6 = m * 2^e with m in [0.5, 1), so 2^e >= top / 6 (top = 0: 2^-127)
        m, e = torch.frexp(top / 6)
        exponent = torch.where(top > 0, torch.where(m == 0.5, e - 1, e), -127).clamp(-127, 127)
        scales = (exponent + 127).to(torch.uint8)
        v = torch.ldexp(g, -exponent.unsqueeze(-1))
        values = torch.tensor(E2M1_VALUES, device=w.device)
        q = torch.bucketize(v.abs(), (values[1:] + values[:-1]) / 2).to(torch.uint8)
        q = q | (v < 0).to(torch.uint8) << 3
    elif zeros:
        lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
        scales = torch.where(hi > lo, (hi - lo) / 15, 1).to(torch.bfloat16)
        s = scales.float().unsqueeze(-1)
        z = torch.round(-lo.unsqueeze(-1) / s).clamp(0, 15)
        q = (torch.round(g / s) + z).clamp(0, 15).to(torch.uint8)
        zero = z.squeeze(-1).to(torch.uint8)
    else:
        top = g.abs().amax(-1)
        scales = torch.where(top > 0, top / 7, 1).to(torch.bfloat16)
        q = (torch.round(g / scales.float().unsqueeze(-1)) + 8).clamp(0, 15).to(torch.uint8)
    q = q.flatten(-2)
    return W4Weights(q[..., 0::2] | q[..., 1::2] << 4, scales, zero, w_format, group_size)
