"""The gated activation as e4m3 rows against its formula in 64 bits."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
import rows_reference as ref
from rows_reference import F32

pytestmark = pytest.mark.gpu

REL = 16 * F32  # exponential, quotient and products of a few half steps each


def call(G, q, s, rows, El=3, max_rows=None, stream=None):
    offsets = torch.full((El + 1,), rows, dtype=torch.int32, device="cuda")
    offsets[0] = 0
    c = ep.ep_config(1, 0, El, 1, 1, 1, 64, 64, 128, ep.EP_FP8_1D2D, -1, 0)
    a = ep.ep_swiglu_e4m3_args(G=ep.ptr(G), q=ep.ptr(q), q_scales=ep.ptr(s), expert_offsets=ep.ptr(offsets),
                               max_rows=max_rows or G.shape[0], inter=G.shape[1] // 2)
    ep.ep_swiglu_e4m3(c, a, stream)
    return offsets


@pytest.mark.parametrize("rows,inter", [(1, 8), (1, 128), (3, 136), (64, 2048), (1, 14336), (1000, 1000),
                                        (4097, 256), (2, 120), (333, 264)])
def test_rows(rows, inter):
    gen = torch.Generator().manual_seed(rows + inter)
    over = 5  # rows that are not there
    G = (2 * torch.randn(rows + over, 2 * inter, generator=gen)).cuda().bfloat16()
    q = torch.full((rows + over, inter), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + over, (inter + 127) // 128), 7.0, device="cuda")
    call(G, q, s, rows)
    torch.cuda.synchronize()
    ref.check_e4m3(q[:rows].view(torch.float8_e4m3fn), s[:rows], ref.swiglu(G[:rows]), REL)
    assert (q[rows:] == 0x5A).all() and (s[rows:] == 7).all()


@pytest.mark.parametrize("rows,max_rows", [(0, 16), (-4, 16), (40, 16)])
def test_counts_outside_the_rows(rows, max_rows):
    G = torch.ones(48, 256, device="cuda").bfloat16()
    q = torch.full((48, 128), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((48, 1), 7.0, device="cuda")
    call(G, q, s, rows, max_rows=max_rows)
    torch.cuda.synchronize()
    there = min(max(rows, 0), max_rows)
    assert (s[:there] != 7).all() and (s[there:] == 7).all() and (q[there:] == 0x5A).all()


def test_extremes():
    """Groups of zeros, of what is too small for a scale, with infinities and NaN."""
    I = 128 * 6
    G = torch.randn(3, 2 * I, generator=torch.Generator().manual_seed(0)).cuda().bfloat16()
    G[0, :128] = 0                      # zeros
    G[0, 128:256] = 2.0 ** -70          # products of 2^-131 and less
    G[0, I + 128:I + 256] = 2.0 ** -60
    G[0, 300] = torch.nan
    G[0, 400] = torch.inf
    G[0, I + 520] = -torch.inf
    G[1, :I] = -200.0                   # SiLU of -200 is no fp32 number: 0
    q = torch.zeros(3, I, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(3, 6, device="cuda")
    call(G, q, s, 3)
    torch.cuda.synchronize()
    assert torch.equal(s[0].isnan().cpu(), torch.tensor([False, False, True, True, True, False]))
    v = ref.swiglu(G)
    v[1] = 0
    ref.check_e4m3(q, s, v, REL)
    assert (q[1].float() == 0).all()


def test_past_31_bits():
    rows, I = 600000, 2048  # 2.4e9 values of G
    G = torch.zeros(rows, 2 * I, dtype=torch.bfloat16, device="cuda")
    G[-2:] = torch.randn(2, 2 * I, generator=torch.Generator().manual_seed(1)).cuda().bfloat16()
    q = torch.zeros(rows, I, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(rows, I // 128, device="cuda")
    call(G, q, s, rows)
    ref.check_e4m3(q[-2:], s[-2:], ref.swiglu(G[-2:]), REL)
    assert (s[:-2] == ref.TINY).all()


# rows of several chunks of a block's threads, fewer and more of them than blocks; the last chunk's and
# the last group's ends
@pytest.mark.parametrize("rows,inter", [(5000, 1032), (70, 14344), (3001, 1352), (641, 4104), (20000, 136),
                                        (9, 65544)])
def test_rows_of_several_chunks(rows, inter):
    gen = torch.Generator(device="cuda").manual_seed(rows + inter)
    G = (2 * torch.randn(rows + 2, 2 * inter, generator=gen, device="cuda")).bfloat16()
    q = torch.full((rows + 2, inter), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 2, (inter + 127) // 128), 7.0, device="cuda")
    call(G, q, s, rows)
    torch.cuda.synchronize()
    ref.check_e4m3(q[:rows].view(torch.float8_e4m3fn), s[:rows], ref.swiglu(G[:rows]), REL)
    assert (q[rows:] == 0x5A).all() and (s[rows:] == 7).all()
