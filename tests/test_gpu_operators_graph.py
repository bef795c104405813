"""The router, the 4-bit layer, the combine and the gradients captured once in a CUDA graph: a replay
on other logits and tokens gives the bits of the calls made one by one."""

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4

pytestmark = pytest.mark.gpu

R, EL, K_TOP, H, I = 2, 8, 3, 256, 128


def build(tokens, fmt, seed):
    gen = torch.Generator().manual_seed(seed)
    s = EpSystem(R, EL, K_TOP, tokens, K=I, N=H)
    t = dict(x=[], logits=[], dout=[], dgates=[], dlogits=[])
    for r in range(R):
        t["x"].append(torch.zeros(tokens, H, dtype=torch.bfloat16, device="cuda"))
        s.set_layer_w4(r, t["x"][r],
                       quantize_w4(torch.randn(EL, 2 * I, H, generator=gen).cuda() / 16, fmt),
                       quantize_w4(torch.randn(EL, H, I, generator=gen).cuda() / 8, fmt))
        t["logits"].append(torch.zeros(tokens, R * EL, device="cuda"))
        t["dout"].append(torch.zeros(tokens, H, dtype=torch.bfloat16, device="cuda"))
        t["dgates"].append(torch.zeros(tokens, K_TOP, device="cuda"))
        t["dlogits"].append(torch.zeros(tokens, R * EL, device="cuda"))
    return s, t


def fill(t, seed):
    gen = torch.Generator().manual_seed(seed)
    for name in ("x", "logits", "dout"):
        for v in t[name]:
            v.copy_(torch.randn(v.shape, generator=gen))


def step(s, t, stream):
    for r in range(R):
        s.route(r, t["logits"][r], score=ep.EP_SCORE_SIGMOID, n_groups=4, topk_groups=2, group_top=2,
                stream=stream)
    for r in range(R):
        s.plan(r, stream=stream)
        s.layer_forward_w4(r, epoch=1, stream=stream)
    for r in range(R):
        s.combine(r, epoch=1, stream=stream, overlap=ep.EP_OVERLAP_ANY)
        s.combine_backward(r, t["dout"][r], dgates=t["dgates"][r], stream=stream)
        s.route_backward(r, t["dgates"][r], t["dlogits"][r], stream=stream)


def results(s, t):
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all(), s.status_words()
    return [v.float().cpu().numpy() for v in [s.topk, *s.gates, *s.out, *t["dgates"], *t["dlogits"]]]


@pytest.mark.parametrize("tokens,fmt", [(1, ep.EP_W4_INT), (40, ep.EP_W4_E2M1), (150, ep.EP_W4_INT),
                                        (150, ep.EP_W4_E2M1)])
def test_replays_give_the_bits_of_single_calls(tokens, fmt):
    s, t = build(tokens, fmt, 5)
    stream = torch.cuda.Stream()
    fill(t, 1)
    torch.cuda.synchronize()
    step(s, t, stream)  # once outside, on the stream that captures
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(s, t, torch.cuda.current_stream())
    one, u = build(tokens, fmt, 5)
    for seed in (2, 3, 4):
        fill(t, seed)
        fill(u, seed)
        for a in (s, one):
            for b in a.recv:
                b.fill_(0xFF)
            for c in a.counts:
                c.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        step(one, u, torch.cuda.current_stream())
        for a, b in zip(results(s, t), results(one, u)):
            np.testing.assert_array_equal(a, b)
