"""quantize_w4 of weights that do not lie contiguously: its tensors go to the kernels by address, so
what counts is the raw memory, the same as for a contiguous copy of the weights."""

import pytest
import torch

from moe_expert_gemm_gb300 import EP_W4_E2M1, EP_W4_INT
from moe_expert_gemm_gb300.w4 import quantize_w4


def raw(t):
    """The bytes from the tensor's address on, whatever its strides say."""
    t8 = t.view(torch.uint8) if t.dtype != torch.uint8 else t
    return torch.as_strided(t8, (t8.numel(),), (1,), t8.storage_offset())


def views(w):
    E, N, K = w.shape
    padded = torch.full((E, N + 3, K + 5), 9.0)
    padded[:, 1:N + 1, 2:K + 2] = w
    return {"stored [E][K][N]": w.transpose(1, 2).contiguous().transpose(1, 2),
            "stored [N][E][K]": w.transpose(0, 1).contiguous().transpose(0, 1),
            "cut out": padded[:, 1:N + 1, 2:K + 2],
            "every other row": torch.stack((w, w + 1), 2).flatten(1, 2)[:, ::2]}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt,group,zeros", [(EP_W4_INT, 32, True), (EP_W4_INT, 64, False),
                                             (EP_W4_E2M1, 32, False)])
def test_any_strides_give_the_same_memory(fmt, group, zeros, dtype):
    w = torch.randn(2, 6, 128, generator=torch.Generator().manual_seed(group)).to(dtype)
    want = quantize_w4(w, fmt, group, zeros)
    for name, view in views(w.float()).items():
        view = view if dtype == torch.float32 else view.to(dtype)
        assert torch.equal(view, w)
        got = quantize_w4(view, fmt, group, zeros)
        for field in ("codes", "scales", "zeros"):
            a, b = getattr(want, field), getattr(got, field)
            assert (a is None) == (b is None)
            if a is not None:
                assert b.is_contiguous() and torch.equal(raw(a), raw(b)), (name, field)


def test_one_row_for_all():
    """An expanded weight row."""
    row = torch.randn(1, 1, 64, generator=torch.Generator().manual_seed(1))
    want = quantize_w4(row.repeat(2, 3, 1))
    got = quantize_w4(row.expand(2, 3, 64))
    for field in ("codes", "scales", "zeros"):
        assert torch.equal(raw(getattr(want, field)), raw(getattr(got, field)))
