"""EpSystem's calls on streams other than torch's current one. What a call allocates for itself
has to be filled on the stream the call goes to: here the current stream is kept busy, so
that anything left on it would land long after the kernels and wipe out what they wrote."""

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
import operator_reference as ref
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4

pytestmark = pytest.mark.gpu

R, EL, K_TOP, T, H, I = 2, 4, 3, 33, 128, 64
BUSY = 200_000_000  # cycles, about a tenth of a second


def layer(seed):
    gen = torch.Generator().manual_seed(seed)
    s = EpSystem(R, EL, K_TOP, T, K=I, N=H)
    logits = []
    for r in range(R):
        s.set_layer_w4(r, torch.randn(T, H, generator=gen).cuda().bfloat16(),
                       quantize_w4(torch.randn(EL, 2 * I, H, generator=gen).cuda() / 16),
                       quantize_w4(torch.randn(EL, H, I, generator=gen).cuda() / 8))
        logits.append(torch.randn(T, R * EL, generator=gen).cuda())
    return s, logits


def step(s, logits, streams, ints=False):
    """One pass of all ranks, each rank's calls on its own stream, ordered by events."""
    of = [st.cuda_stream if ints else st for st in streams]

    def meet():
        marks = [st.record_event() for st in streams]
        for st in streams:
            for m in marks:
                st.wait_event(m)

    for r in range(R):
        s.route(r, logits[r], stream=of[r])
    meet()
    for r in range(R):
        s.plan(r, stream=of[r])
        s.layer_forward_w4(r, epoch=1, stream=of[r])
    meet()
    for r in range(R):
        s.combine(r, epoch=1, stream=of[r])


def results(s):
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all(), s.status_words()
    plans = [{k: v.cpu().numpy() for k, v in p.items() if torch.is_tensor(v)} for p in s.plans]
    return ([s.topk.cpu().numpy()] + [g.cpu().numpy() for g in s.gates] +
            [o.view(torch.int16).cpu().numpy() for o in s.out], plans)


@pytest.mark.parametrize("ints", [False, True])
@pytest.mark.parametrize("n_streams", [1, 2])
def test_calls_beside_a_busy_current_stream(n_streams, ints):
    s, logits = layer(1)
    here = torch.cuda.current_stream()
    step(s, logits, [here] * R)
    want, want_plans = results(s)
    for r in range(R):
        ids = [ref.chosen(l, np.zeros(l.size, bool), "softmax", None, K_TOP)
               for l in logits[r].double().cpu().numpy()]
        np.testing.assert_array_equal(want[0][r], ids)
    s, logits = layer(1)
    side = [torch.cuda.Stream() for _ in range(n_streams)] * (R // n_streams)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    step(s, logits, side, ints)
    busy = not here.query()
    for st in side:
        st.synchronize()
    got, plans = results(s)
    assert busy, "the current stream was idle: nothing was shown"
    for a, b in zip(want, got):
        np.testing.assert_array_equal(a, b)
    for p, q in zip(want_plans, plans):
        for name in p:
            m = int(p["m_total"][0]) if name in ("src_info", "gather_idx") else None
            np.testing.assert_array_equal(p[name][:m], q[name][:m], err_msg=name)


def test_calls_without_a_stream_go_to_the_default_one():
    """Inside another current stream: the default stream's kernels follow their own fills."""
    s, logits = layer(2)
    step(s, logits, [torch.cuda.default_stream()] * R)
    want, _ = results(s)
    s, logits = layer(2)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(BUSY)
        for r in range(R):
            s.route(r, logits[r])
        for r in range(R):
            s.plan(r)
            s.layer_forward_w4(r, epoch=1)
        for r in range(R):
            s.combine(r, epoch=1)
    got, _ = results(s)
    for a, b in zip(want, got):
        np.testing.assert_array_equal(a, b)
