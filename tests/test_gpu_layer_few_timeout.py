"""Waits of the layer of a few tokens that run out: limits shorter than the first bytes take to come. The call
reports it and ends, and once the workspace is zeroed the next one is right."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300.system import STATUS_FEW, EpSystem
from test_gpu_layer_few import Few

pytestmark = pytest.mark.gpu


def limited(f, ns):
    a = ep.ep_layer_few_args(x=ep.ptr(f.x), x_scales=ep.ptr(f.xs), topk_ids=ep.ptr(f.ids), gates=ep.ptr(f.gates),
                             W1=ep.ptr(f.W1), w1_scales=ep.ptr(f.w1s), W2=ep.ptr(f.W2), w2_scales=ep.ptr(f.w2s),
                             out=ep.ptr(f.out), workspace=ep.ptr(f.work), workspace_bytes=f.size,
                             status=ep.ptr(f.status), timeout_ns=ns)
    ep.ep_layer_few(f.cfg, a)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 20, 64])
def test_limits_that_run_out(T, fp8):
    f = Few(T, 8, 4, 2048, 1024, fp8=fp8, seed=T)
    seen = 0
    for i in range(8):  # (also on counters that the call before left)
        f.status.zero_()
        limited(f, 1)
        torch.cuda.synchronize()
        assert int(f.status) in (0, ep.EP_STATUS_TIMEOUT)
        seen += int(f.status) == ep.EP_STATUS_TIMEOUT
    assert seen > 0
    assert (f.work[f.size:] == 0x5A).all()
    f.work[:f.size] = 0
    f.status.zero_()
    limited(f, 1_000_000_000)
    f.check()


def test_the_systems_limit_and_reset():
    T, E, H, I = 16, 8, 2048, 1024
    s = EpSystem(1, E, 2, T, K=I, N=H, timeout_ns=1)
    gen = torch.Generator().manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen).cuda().bfloat16()
    s.set_layer_few(0, rand(E, 2 * I, H) * H ** -0.5, rand(E, H, I) * I ** -0.5)
    s.route(0, torch.randn(T, E, generator=gen).cuda())
    x, out, again = rand(T, H), rand(T, H), rand(T, H)
    torch.cuda.synchronize()
    for i in range(8):
        s.layer_few(0, x, out)
    torch.cuda.synchronize()
    assert s.status_words()[STATUS_FEW] == ep.EP_STATUS_TIMEOUT
    at = s.layer_few_ops[0]["workspace"].data_ptr()
    s.status.zero_()
    s.timeout_ns = 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.reset_layer_few(0, stream=side)
    s.layer_few(0, x, out, stream=side)
    s.layer_few(0, x, again, stream=side)
    torch.cuda.synchronize()
    assert s.layer_few_ops[0]["workspace"].data_ptr() == at
    assert (s.status_words() == 0).all()
    fresh = EpSystem(1, E, 2, T, K=I, N=H)
    ops = s.layer_few_ops[0]
    fresh.set_layer_few(0, ops["W1"], ops["W2"])
    fresh.topk, fresh.gates = s.topk, s.gates
    want = torch.zeros_like(out)
    fresh.layer_few(0, x, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(again, want)
