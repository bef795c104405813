"""Of the workspace of the layer of a few tokens only the counters at its head have to be zero."""

import os
import re

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300.system import EpSystem
from test_gpu_layer_few import Few


def test_the_headers_constant():
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_ep.h")
    assert int(re.search(r"#define EP_FEW_COUNTER_BYTES (\d+)", open(header).read()).group(1)) == ep.EP_FEW_COUNTER_BYTES


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 256, 1024), (20, 8, 3, 512, 640), (64, 6, 3, 1024, 384)])
def test_the_rest_may_hold_anything(T, E, k, H, I, fp8):
    f = Few(T, E, k, H, I, fp8=fp8, seed=T)
    f.work[:f.size] = 0xFF
    f.work[:ep.EP_FEW_COUNTER_BYTES] = 0
    f.call()
    f.check()


@pytest.mark.gpu
def test_the_systems_workspace():
    """On memory that somebody else has used."""
    T, E, H, I = 33, 8, 512, 256
    s = EpSystem(1, E, 2, T, K=I, N=H)
    gen = torch.Generator().manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen).cuda().bfloat16()
    W1, W2, x = rand(E, 2 * I, H) * H ** -0.5, rand(E, H, I) * I ** -0.5, rand(T, H)
    s.route(0, torch.randn(T, E, generator=gen).cuda())
    outs = []
    for fill in (0, 0xFF):
        s.layer_few_ops[0] = None
        used = [torch.full((ep.ep_layer_few_sizes(s.cfg(0)),), fill, dtype=torch.uint8, device="cuda")
                for _ in range(4)]
        places = {u.data_ptr() for u in used}
        del used
        s.set_layer_few(0, W1, W2)
        workspace = s.layer_few_ops[0]["workspace"]
        assert workspace.data_ptr() in places and (workspace[:ep.EP_FEW_COUNTER_BYTES] == 0).all()
        outs.append(torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"))
        s.layer_few(0, x, outs[-1])
        torch.cuda.synchronize()
        del workspace
    assert torch.equal(outs[0], outs[1]) and outs[0].isfinite().all()
    assert (s.status_words() == 0).all()
