"""The whole fp8 layer (norm to e4m3, router, plan, dispatch, products, activation to e4m3, send, combine) at widths
and row counts of real use, against its formula in 64 bits."""

import math

import pytest
import torch

import rows_reference as ref
from moe_expert_gemm_gb300.system import EpSystem
from rows_reference import BF16, E4M3, F32

pytestmark = pytest.mark.gpu


def weights(E, N, K, gen):
    """e4m3 codes and the scales of 128 x 128 blocks of N(0, 1 / K) values."""
    w = torch.randn(E, N // 128, 128, K // 128, 128, generator=gen, device="cuda") * K ** -0.5
    s = w.abs().amax((2, 4)) / 448
    return (w / s[:, :, None, :, None]).view(E, N, K).to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("T,E,k,H,I", [(300, 6, 3, 7168, 2048), (1500, 4, 2, 2048, 1408), (9, 8, 4, 4096, 2048)])
def test_layer(T, E, k, H, I):
    gen = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    s = EpSystem(1, E, k, T, K=I, N=H, dtype="fp8_1d2d")
    x, residual, weight = rand(T, H).bfloat16(), rand(T, H), 1 + 0.2 * rand(H)
    y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    q, qs = torch.zeros(T, H, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(T, H // 128, device="cuda")
    W1, s1 = weights(E, 2 * I, H, gen)
    W2, s2 = weights(E, H, I, gen)
    s.add_rmsnorm(0, x, weight, residual=residual, sum=residual, y=y, q=q, q_scales=qs)
    s.route(0, y.float() @ (rand(H, E) * H ** -0.5))
    s.plan(0)
    s.set_layer_fp8(0, q, qs, W1, s1, W2, s2)
    for epoch in (1, 2):
        s.layer_forward_fp8(0, epoch)
        s.combine(0, epoch)
        torch.cuda.synchronize()
        assert (s.status_words() == 0).all()
        out = s.out[0].clone() if epoch == 1 else out
    assert torch.equal(out, s.out[0])

    x64, want = ref.wide(q, qs), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    bound, size = torch.zeros_like(want), torch.zeros_like(want)
    for e in range(E):
        t, j = torch.nonzero(s.topk[0] == e, as_tuple=True)
        w = ref.wide_blocks(W1[e], s1[e])
        gu = x64[t] @ w.T
        # the up/gate rows: sums of H values, rounded to bf16
        err = BF16 * gu.abs() + 2 * (H + 8) * F32 * (x64[t].abs() @ w.abs().T)
        gate, up, eg, eu = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
        a = ref.swiglu(gu)
        # |SiLU'| <= 1.1; then half a step of e4m3
        ea = 1.1 * eg * (up.abs() + eu) + (gate * torch.sigmoid(gate)).abs() * eu + 16 * F32 * a.abs()
        ea = ea + E4M3 * (a.abs() + ea) + 2.0 ** -10 * ref.scales(a).repeat_interleave(128, 1)
        w, g = ref.wide_blocks(W2[e], s2[e]), s.gates[0][t, j].double()[:, None]
        row = a @ w.T
        want.index_add_(0, t, g * row)
        # the rows: sums of I values, rounded to bf16, times the gates
        off = ea @ w.abs().T + 2 * (I + 8) * F32 * (a.abs() @ w.abs().T)
        bound.index_add_(0, t, g * (off + BF16 * (row.abs() + off)))
        size.index_add_(0, t, g * row.abs())
    bound += (k + 2) * F32 * size
    got = out.double()
    assert ((got - want).abs() <= BF16 * (want.abs() + bound) + bound).all()
    # As a whole: the codes' roundings are as good as independent, at most E4M3 of a value and evenly spread, of
    # a root mean square of E4M3 / sqrt(3) at most; bf16 roundings of the up/gate rows (two), rows and out
    # beside it.
    off = (got - want).norm() / want.norm()
    assert off <= E4M3 / math.sqrt(3) + 4 * BF16
    assert off >= E4M3 / 16  # (and the activation did go through 8 bits)
