"""The combine that does not wait (EP_OVERLAP_INPUTS_READY) behind kernels that write none of its
inputs, where the kernel before those writes the gates: that one has to have ended."""

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4

pytestmark = pytest.mark.gpu

E, K_TOP, T, N = 256, 8, 40000, 64


def config(experts, top_k, tokens, K, N):
    return ep.ep_config(n_ranks=1, my_rank=0, n_local_experts=experts, top_k=top_k,
                        num_tokens=tokens, max_tokens_per_rank=max(tokens, 1), K=K, N=N,
                        msg_bytes=2 * N, dtype=ep.EP_BF16, send_warps=-1, signal_mode=0)


def products(rows):
    """A call of the 4-bit products of its own, of the form for `rows` rows an expert."""
    w = quantize_w4(torch.randn(1, 96, 256, generator=torch.Generator().manual_seed(1)).cuda() / 16)
    conf = config(1, 1, rows, 256, 96)
    n = ep.ep_matvec_w4_sizes(conf)
    keep = dict(x=torch.ones(rows, 256, dtype=torch.bfloat16, device="cuda"), w=w,
                off=torch.tensor([0, rows], dtype=torch.int32, device="cuda"),
                C=torch.zeros(rows, 96, dtype=torch.bfloat16, device="cuda"),
                ws=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    a = ep.ep_w4_args(A=ep.ptr(keep["x"]), W=ep.ptr(w.codes), w_scales=ep.ptr(w.scales),
                      w_zeros=ep.ptr(w.zeros), w_format=w.w_format, group_size=w.group_size,
                      expert_offsets=ep.ptr(keep["off"]), max_rows=rows, C=ep.ptr(keep["C"]),
                      workspace=ep.ptr(keep["ws"]), workspace_bytes=n, status=ep.ptr(keep["status"]))
    return lambda st: ep.ep_matvec_w4(conf, a, st), keep


def small_route():
    keep = dict(l=torch.randn(3, 32, device="cuda"), i=torch.zeros(3, 2, dtype=torch.int32, device="cuda"),
                g=torch.zeros(3, 2, device="cuda"), d=torch.zeros(3, 32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    conf = config(32, 2, 3, 64, 64)
    a = ep.ep_route_args(logits=ep.ptr(keep["l"]), scale=1.0, topk_ids=ep.ptr(keep["i"]),
                         gates=ep.ptr(keep["g"]))
    b = ep.ep_route_backward_args(logits=ep.ptr(keep["l"]), scale=1.0, topk_ids=ep.ptr(keep["i"]),
                                  dgates=ep.ptr(keep["g"]), dlogits=ep.ptr(keep["d"]),
                                  status=ep.ptr(keep["status"]))
    return conf, a, b, keep


@pytest.mark.parametrize("between", ["products of one row", "products of 40 rows", "route",
                                     "route backward", "combine backward"])
def test_gates_of_the_kernel_before_the_previous_one(between):
    gen = torch.Generator().manual_seed(3)
    s = EpSystem(1, E, K_TOP, T, K=64, N=N)
    s.recv[0].view(torch.bfloat16).copy_(torch.randn(T * K_TOP * N, generator=gen))
    s.counts[0][E] = 1  # the only source rank's flag, of epoch 1
    logits = torch.randn(T, E, generator=gen).cuda()
    if between.startswith("products"):
        call, keep = products(1 if "one" in between else 40)
    elif between.startswith("route"):
        conf, a, b, keep = small_route()
        call = lambda st: ep.ep_route(conf, a, st) if between == "route" else ep.ep_route_backward(conf, b, st)
    else:
        conf = config(4, 2, 2, 64, 64)
        keep = dict(rows=torch.ones(2 * 2 * 64, dtype=torch.bfloat16, device="cuda"),
                    dout=torch.ones(2, 64, dtype=torch.bfloat16, device="cuda"),
                    dg=torch.zeros(2, 2, device="cuda"))
        a = ep.ep_combine_backward_args(recv_buf=ep.ptr(keep["rows"]), dout=ep.ptr(keep["dout"]),
                                        dgates=ep.ptr(keep["dg"]))
        call = lambda st: ep.ep_combine_backward(conf, a, st)
    s.route(0, logits, n_groups=8, topk_groups=1)  # a call of some hundred us
    s.combine(0, epoch=1)
    torch.cuda.synchronize()
    want, gates = s.out[0].clone(), s.gates[0].clone()
    assert torch.isfinite(want.float()).all()
    for overlap in (ep.EP_OVERLAP_INPUTS_READY, ep.EP_OVERLAP_ANY):
        for _ in range(5):
            s.gates[0].fill_(float("nan"))
            s.out[0].fill_(77.0)
            torch.cuda.synchronize()
            s.route(0, logits, n_groups=8, topk_groups=1)
            call(None)
            s.combine(0, epoch=1, overlap=overlap)
            torch.cuda.synchronize()
            assert torch.equal(s.gates[0], gates)
            assert torch.equal(s.out[0], want), (s.out[0] != want).any(1).sum()
    assert (s.status_words() == 0).all()
    if "status" in keep:
        assert keep["status"].item() == 0


@pytest.mark.parametrize("signal_mode", [0, 1])
@pytest.mark.parametrize("top_k", [2, 3])
def test_a_kernel_behind_the_combine_that_does_not_wait(top_k, signal_mode):
    """A long kernel, a short combine of other buffers that does not wait for it, and a kernel that
    reads what the long one writes: it has to come after both."""
    gen = torch.Generator().manual_seed(4)
    s = EpSystem(1, E, K_TOP, T, K=64, N=N)
    logits = torch.randn(T, E, generator=gen).cuda()
    dout = torch.randn(T, N, generator=gen).cuda().bfloat16()
    drows = torch.zeros(T, K_TOP, N, dtype=torch.bfloat16, device="cuda")
    small = EpSystem(1, 4, top_k, 3, K=64, N=64, signal_mode=signal_mode)
    small.recv[0].view(torch.bfloat16).copy_(torch.randn(3 * top_k * 64, generator=gen))
    small.counts[0].fill_(1 << 32 if signal_mode else 1)  # every signal of epoch 1 is there
    small.set_routing(np.tile(np.arange(top_k), (1, 3, 1)))
    small.set_gates(0, np.ones((3, top_k)))
    for overlap in (ep.EP_OVERLAP_NONE, ep.EP_OVERLAP_INPUTS_READY, ep.EP_OVERLAP_ANY):
        for _ in range(5):
            s.route(0, logits, n_groups=8, topk_groups=1)
            s.gates[0].fill_(float("nan"))
            small.out[0].fill_(77.0)
            drows.fill_(55.0)
            torch.cuda.synchronize()
            s.route(0, logits, n_groups=8, topk_groups=1)
            small.combine(0, epoch=1, overlap=overlap)
            s.combine_backward(0, dout, drows=drows)
            torch.cuda.synchronize()
            want = (s.gates[0][:, :, None] * dout[:, None, :].float()).to(torch.bfloat16)
            assert torch.equal(drows, want), (drows != want).any(2).sum()
            rows = small.recv[0].view(torch.bfloat16).view(3, top_k, 64).float().sum(1)
            assert torch.allclose(small.out[0].float(), rows, rtol=2.0 ** -8, atol=1e-6)
    assert (s.status_words() == 0).all() and (small.status_words() == 0).all()
