"""A step of a rank group without tokens through the router and the 4-bit layer: nothing to
compute, but every call is made, and the flags have to come."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [ep.EP_W4_INT, ep.EP_W4_E2M1])
def test_no_tokens(fmt):
    R, El, k, H, I = 2, 3, 2, 128, 64
    gen = torch.Generator().manual_seed(0)
    s = EpSystem(R, El, k, 0, K=I, N=H, max_tokens=4)
    for r in range(R):
        s.set_layer_w4(r, torch.zeros(4, H, dtype=torch.bfloat16, device="cuda"),
                       quantize_w4(torch.randn(El, 2 * I, H, generator=gen).cuda(), fmt),
                       quantize_w4(torch.randn(El, H, I, generator=gen).cuda(), fmt))
        s.route(r, torch.zeros(0, R * El, device="cuda"))
    for r in range(R):
        s.plan(r)
        s.layer_forward_w4(r, epoch=3)
    for r in range(R):
        s.combine(r, epoch=3)
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all(), s.status_words()
    for r in range(R):
        assert (s.counts[r][El * R:] == 3).all()


def test_gradients_of_no_tokens():
    R, El, k, H = 2, 3, 2, 128
    s = EpSystem(R, El, k, 0, K=64, N=H, max_tokens=4)
    empty = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")
    for r in range(R):
        s.route(r, empty(0, R * El))
        s.combine_backward(r, empty(0, H, dtype=torch.bfloat16), dgates=empty(0, k))
        s.combine_backward(r, empty(0, H, dtype=torch.bfloat16), drows=s.recv[r])
        s.route_backward(r, empty(0, k), empty(0, R * El))
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all()
    assert all((b == 0xFF).all() for b in s.recv)
