"""SiLU of gates down to where e^-x leaves fp32 (the last bf16 gate is -88.5): values of 2^-120 and so, which
large factors and the scales of 8-bit rows bring back into sight."""

import pytest
import torch

import rows_reference as ref
from rows_reference import BF16, E4M3, F32
from test_gpu_layer_few import Few
from test_gpu_swiglu_e4m3 import REL, call

pytestmark = pytest.mark.gpu

GATES = [-86.0, -87.0, -87.5, -88.0, -88.5]


@pytest.mark.parametrize("up", [1.0, 2.0 ** -3, 2.0 ** 40, 2.0 ** 120])
def test_activation_to_8_bits(up):
    I = 128 * len(GATES)
    G = torch.empty(3, 2 * I)
    G[:, :I] = torch.tensor(GATES).repeat_interleave(128)  # a group of each
    G[:, I:] = up * (1 + torch.rand(3, I, generator=torch.Generator().manual_seed(0)))
    G[2, :I] = torch.tensor(GATES).repeat(128)             # and mixed
    G = G.bfloat16().cuda()
    q = torch.zeros(3, I, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(3, len(GATES), device="cuda")
    call(G, q, s, 3)
    torch.cuda.synchronize()
    v = ref.swiglu(G)
    ref.check_e4m3(q, s, v, REL)
    # seen at all: every group's largest value is more than a step of the smallest scale
    assert (ref.groups(v).abs().amax(-1) >= 2 * ref.TINY).all()
    assert (ref.groups(q.double()).abs().amax(-1) > 0).all()


def test_behind_the_end():
    """Where e^-x is infinite in fp32, SiLU is 0, whatever it meets."""
    G = torch.full((1, 256), -89.0)
    G[0, 128:] = 2.0 ** 120
    q = torch.zeros(1, 128, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(1, 1, device="cuda")
    call(G.bfloat16().cuda(), q, s, 1)
    torch.cuda.synchronize()
    assert (q.float() == 0).all() and (s == ref.TINY).all()


def test_products_near_the_largest():
    """Finite values of any size are no infinity, whatever the gate or the factor alone comes to; groups
    beside them are not touched."""
    I = 128 * 6
    G = torch.randn(2, 2 * I, generator=torch.Generator().manual_seed(1))
    G[0, 5], G[0, I + 5] = 2.0 ** 127, 1.5      # gate, product past 2^126
    G[0, 133], G[0, I + 133] = 3.0, 2.0 ** 126
    G[0, 261], G[0, I + 261] = 2.0 ** 64, 2.0 ** 63
    G[0, 389], G[0, I + 389] = 2.0 ** 127, 2.0 ** -60
    G[0, 517], G[0, I + 517] = 2.0 ** 100, 2.0 ** 28  # an infinity
    G = G.bfloat16().cuda()
    q = torch.zeros(2, I, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(2, 6, device="cuda")
    call(G, q, s, 2)
    torch.cuda.synchronize()
    v = ref.swiglu(G)
    v[0, 517] = torch.inf  # (fp32: 2^128)
    ref.check_e4m3(q, s, v, REL)
    assert s.isnan().sum() == 1 and s[0, 4].isnan()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gate", GATES)
def test_layer_of_a_few_tokens(fp8, gate):
    """One expert whose gates are all `gate` and whose second matrix is of 2^100."""
    H = I = 128
    f = Few(2, 1, 1, H, I, fp8=fp8)
    f.gates.fill_(1)
    for w in (f.x, f.W1):
        w.copy_(torch.zeros(w.shape))
    f.x[:, :2] = 1
    f.W1[0, :I, 0] = -1 if fp8 else gate
    up = 1 + torch.arange(I) % 8 / 8
    f.W1[0, I:, 1] = up.to(f.W1.dtype).cuda()
    w2 = 1 + torch.randint(0, 8, (H, I), generator=torch.Generator().manual_seed(0)) / 8
    f.W2[0] = (w2 if fp8 else w2 * 2.0 ** 100).to(f.W2.dtype).cuda()
    if fp8:
        f.xs.fill_(1)
        f.w1s.copy_(torch.tensor([-gate, 1.0]).view(1, 2, 1))
        f.w2s.fill_(2.0 ** 100)
    f.call()
    torch.cuda.synchronize()
    assert int(f.status) == 0
    x = torch.tensor(gate, dtype=torch.float64)
    a = (x * torch.sigmoid(x) * up.double())  # (the first product has one term a value: exact)
    step = E4M3 * a.abs() + 2.0 ** -10 * ref.scales(a[None])[0] if fp8 else BF16 * a.abs()
    want = 2.0 ** 100 * (w2.double() @ a)
    off = 2.0 ** 100 * (w2.double() @ (step + (REL + (I + 8) * F32) * a.abs()))
    got = f.out[0].double().cpu()
    assert (got != 0).all()
    assert ((got - want).abs() <= BF16 * (want.abs() + off) + off).all()
    assert torch.equal(f.out[0], f.out[1])


@pytest.mark.parametrize("gate", [-89.0, -200.0, -2.0 ** 100])
def test_layer_of_a_few_tokens_behind_the_end(gate):
    f = Few(2, 1, 1, 128, 128)
    f.gates.fill_(1)
    f.x[:, 0] = 1
    f.W1[0, :128] = 0
    f.W1[0, :128, 0] = gate
    f.W2.fill_(2.0 ** 100)
    f.call()
    torch.cuda.synchronize()
    assert int(f.status) == 0 and (f.out == 0).all()
