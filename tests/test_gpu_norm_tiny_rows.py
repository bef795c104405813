"""The norm's gradient at eps = 0 for rows whose r^2 leaves fp32 (r about 2^66): finite where the gradient
is, r times dy in size."""

import pytest
import torch

import rows_reference as ref
from rows_reference import BF16, F32
from test_gpu_norm import STEP, back_call

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32
# Squares of values of 8 bits and 2^-66 in size are whole multiples of 2^-149: exact, as are their sums in
# 24 bits to within the steps of any row. Their mean is one of fp32's subnormal numbers, to within 2^-150 of
# 2^-132 or more: 2^-18, in r half of it, which enters three times.
TINY = 3 * 2.0 ** -19


@pytest.mark.parametrize("n", [256, 203, 2048, 6001])
@pytest.mark.parametrize("h_type", [B, F])
def test_gradient_of_tiny_rows(n, h_type):
    T = 5
    gen = torch.Generator().manual_seed(n)
    sign = torch.randint(0, 2, (T, n), generator=gen) * 2 - 1
    h = ((1 + torch.randint(0, 128, (T, n), generator=gen) / 128) * sign * 2.0 ** -66).to(h_type).cuda()
    dy = torch.randn(T, n, generator=gen).cuda().to(B)
    w = (1 + 0.3 * torch.randn(n, generator=gen)).cuda()
    dh, dx, dw = torch.zeros_like(h), torch.zeros_like(dy), torch.zeros(n, device="cuda")
    back_call(h, dy, w, None, dh, dx, dw, eps=0.0)
    torch.cuda.synchronize()
    want, want_w, size, size_w = ref.norm_backward(h, dy, w, None, 0.0)
    off = (256 * F32 + TINY) * size
    assert want.abs().max() > 2.0 ** 60
    assert ((dh.double() - want).abs() <= STEP[h_type] * (want.abs() + off) + off).all()
    assert ((dx.double() - want).abs() <= BF16 * (want.abs() + off) + off).all()
    assert ((dw.double() - want_w).abs() <= (64 * F32 + TINY) * size_w).all()
