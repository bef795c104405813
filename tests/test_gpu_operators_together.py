"""The router, the 4-bit layer, the combine and their gradients as EpSystem runs them
one after the other, against the 64-bit formulas from the logits to the logits' gradient.

Bounds, with u = 2^-8 for a rounding to bf16 and fp32 sums of K products within K 2^-23 of
the sum of their magnitudes: an activation is off by u of itself plus what the first
product's fp32 errors do to it (|silu'| <= 1.1), a row by u of itself plus sum |w| times
that plus its own fp32 sum, an output by u of itself plus the gates' sum over its rows;
the gates' fp32 error (under 2^-18 of each) is inside the margin of 1 %. dgates sums
|dout| times a row's error; the logits' gradient is taken from the dgates the device
produced, its fp32 steps within 2^-18 of the magnitudes it is summed from."""

import os
import sys

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
import operator_reference as ref
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def dequant(w):
    fmt = "e2m1" if w.w_format == ep.EP_W4_E2M1 else "int4"
    scales = w.scales.cpu().numpy() if fmt == "e2m1" else w.scales.float().cpu().numpy()
    return ref.w4_dequant(w.codes.cpu().numpy(), scales,
                          None if w.zeros is None else w.zeros.cpu().numpy(), fmt, w.group_size)


def row_and_error(x, w1, w2):
    """One expert's row for a token, and how far the device's may be off."""
    H, I = w1.shape[1], w2.shape[1]
    y, size = w1 @ x, np.abs(w1) @ np.abs(x) * H * 2.0 ** -23
    with np.errstate(over="ignore"):
        silu = y[:I] / (1 + np.exp(-y[:I]))
    a = silu * y[I:]
    off = U * np.abs(a) + 1.1 * size[:I] * np.abs(y[I:]) + np.abs(silu) * size[I:]
    row = w2 @ a
    return row, U * np.abs(row) + np.abs(w2) @ off + np.abs(w2) @ np.abs(a) * I * 2.0 ** -23


@pytest.mark.parametrize("fmt,group,tokens", [(ep.EP_W4_E2M1, 32, 24), (ep.EP_W4_INT, 64, 24),
                                              (ep.EP_W4_E2M1, 32, 1), (ep.EP_W4_INT, 32, 70)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_from_logits_and_back(fmt, group, tokens, dtype):
    R, El, k, H, I = 2, 3, 2, 288 if group == 32 else 256, 128
    E = R * El
    gen = torch.Generator().manual_seed(tokens + group)
    s = EpSystem(R, El, k, tokens, K=I, N=H)
    X, W1, W2, logits = [], [], [], []
    for r in range(R):
        X.append(torch.randn(tokens, H, generator=gen).cuda().bfloat16())
        W1.append(quantize_w4(torch.randn(El, 2 * I, H, generator=gen).cuda() / 16, fmt, group))
        W2.append(quantize_w4(torch.randn(El, H, I, generator=gen).cuda() / 8, fmt, group))
        s.set_layer_w4(r, X[r], W1[r], W2[r])
        wide = torch.randn(tokens, E + 3, generator=gen).to(dtype).cuda()  # rows of another stride
        wide[0, 1] = -float("inf")
        logits.append(wide[:, :E])
        s.route(r, logits[r], score=ep.EP_SCORE_SIGMOID, renormalize=True, scale=1.5)
    for r in range(R):
        s.plan(r)
        s.layer_forward_w4(r, epoch=1)
    dgates, dlogits = [], []
    douts = [torch.randn(tokens, H, generator=gen).cuda().bfloat16() for _ in range(R)]
    for r in range(R):
        s.combine(r, epoch=1)
        dgates.append(torch.empty(tokens, k, device="cuda"))
        dlogits.append(torch.empty_like(logits[r], memory_format=torch.contiguous_format))
        s.combine_backward(r, douts[r], dgates=dgates[r])
        s.route_backward(r, dgates[r], dlogits[r])
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all(), s.status_words()

    w1 = np.concatenate([dequant(w) for w in W1])
    w2 = np.concatenate([dequant(w) for w in W2])
    lowest = ref.LOWEST["f32" if dtype == torch.float32 else "bf16"]
    num = lambda t: t.double().cpu().numpy()
    for r in range(R):
        x, l, dout = num(X[r]), num(logits[r]), num(douts[r])
        ids, out = s.topk[r].cpu().numpy(), num(s.out[r])
        for t in range(tokens):
            want = ref.chosen(l[t], l[t] <= lowest, "sigmoid", None, k)
            np.testing.assert_array_equal(ids[t], want)
            g = ref.gates_of(l[t], want, "sigmoid", True, 1.5, lowest)
            rows, offs = zip(*[row_and_error(x[t], w1[e], w2[e]) for e in want])
            y = sum(gj * row for gj, row in zip(g, rows))
            off = sum(gj * o for gj, o in zip(g, offs)) + U * np.abs(y)
            assert (np.abs(out[t] - y) <= 1.01 * off + 1e-30).all()
            dg = num(dgates[r])[t]
            for j in range(k):
                lim = np.abs(dout[t]) @ (offs[j] + np.abs(rows[j]) * H * 2.0 ** -23)
                assert abs(dg[j] - dout[t] @ rows[j]) <= 1.01 * lim
            d, size = ref.gates_backward(l[t], want, dg, "sigmoid", True, 1.5, lowest)
            half = U if dtype == torch.bfloat16 else 0
            assert (np.abs(num(dlogits[r])[t] - d) <= half * np.abs(d) + 2.0 ** -18 * size + 1e-30).all()


@pytest.mark.parametrize("fmt", [ep.EP_W4_E2M1, ep.EP_W4_INT])
def test_example_learns(fmt):
    import train_router
    losses = train_router.train(steps=30, tokens=32, w_format=fmt, log=None)
    assert losses[-1] < losses[0] / 2
