"""The 4-bit layouts on the CPU: what quantize_w4 packs is read back by the reference's
own reading of the layout, as near as the format's steps allow."""

import numpy as np
import pytest
import torch

from moe_expert_gemm_gb300 import EP_W4_E2M1, EP_W4_INT
from moe_expert_gemm_gb300.w4 import quantize_w4
import operator_reference as ref


def read_back(w):
    scales = w.scales.float().numpy() if w.w_format == EP_W4_INT else w.scales.numpy()
    return ref.w4_dequant(w.codes.numpy(), scales, None if w.zeros is None else w.zeros.numpy(),
                          "e2m1" if w.w_format == EP_W4_E2M1 else "int4", w.group_size)


def example(K, seed):
    w = torch.randn(2, 5, K, generator=torch.Generator().manual_seed(seed))
    w[0, 0] *= 1e-3
    w[1, 1, :32] = 0
    w[1, 2] = w[1, 2].abs() + 1
    return w


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
def test_integer_weights_read_back(group, zeros):
    w = example(256, group)
    q = quantize_w4(w, EP_W4_INT, group, zeros)
    assert q.codes.shape == (2, 5, 128) and q.scales.shape == (2, 5, 256 // group)
    assert (q.zeros is not None) == zeros and q.scales.dtype == torch.bfloat16
    # half a step to the nearest code; with a zero point of its own rounded as well, and up
    # to 8 steps of a scale that bf16 makes 2^-9 too small
    step = np.repeat(q.scales.float().numpy(), group, -1)
    assert (abs(read_back(q) - w.numpy()) <= (1.0 if zeros else 0.5) * step + 15 * step / 256).all()


def test_e2m1_weights_read_back():
    w = example(128, 9)
    q = quantize_w4(w, EP_W4_E2M1, 32)
    assert q.scales.dtype == torch.uint8 and q.zeros is None
    step = np.repeat(np.exp2(q.scales.numpy().astype(np.float64) - 127), 32, -1)
    v = w.numpy() / step
    assert (abs(v) <= 6).all()
    top = np.abs(v).reshape(2, 5, 4, 32).max(-1)
    assert ((top > 3) | (top == 0)).all()  # no larger a scale than needed
    gap = np.where(abs(v) <= 2, 0.5, np.where(abs(v) <= 4, 1, 2))
    assert (abs(read_back(q) / step - v) <= gap / 2).all()
    exact = torch.tensor(ref.E2M1[:8].repeat(4)).float()[None]
    assert (read_back(quantize_w4(exact * 0.25, EP_W4_E2M1, 32)) == exact.numpy() * 0.25).all()


@pytest.mark.parametrize("fmt,group,K", [(EP_W4_INT, 16, 64), (EP_W4_INT, 128, 192),
                                         (EP_W4_E2M1, 64, 128), (7, 32, 64)])
def test_refuses_other_layouts(fmt, group, K):
    with pytest.raises(ValueError):
        quantize_w4(torch.zeros(1, K), fmt, group)
