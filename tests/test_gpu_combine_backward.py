"""The combine's gradient on the GPU against the 64-bit definition.

dgates: fp32 sums of N products: |error| <= 2^-24 (N/32 + 32) sum |dout row| (chains of at
most N/32 additions before a tree). drows: the fp32 product rounded to bf16, bit-exact."""

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
import operator_reference as ref

pytestmark = pytest.mark.gpu


def cfg(T, k, N):
    return ep.ep_config(n_ranks=1, my_rank=0, n_local_experts=max(k, 1), top_k=k, num_tokens=T,
                        max_tokens_per_rank=max(T, 1), K=64, N=N, msg_bytes=2 * N,
                        dtype=ep.EP_BF16, send_warps=-1, signal_mode=0)


def inputs(T, k, N, seed):
    rng = np.random.default_rng(seed)
    rows = ref.bf16_round(rng.normal(size=(T, k, N)).astype(np.float32))
    dout = ref.bf16_round(rng.normal(size=(T, N)).astype(np.float32))
    return rows, rng.random((T, k)).astype(np.float32), dout


def run(rows, gates, dout, want_dgates=True, want_drows=True, in_place=False, stream=None):
    T, k, N = rows.shape
    pad = 64  # guard elements behind each output
    bf = lambda x: torch.from_numpy(x).to("cuda", torch.bfloat16)
    r, g, d = bf(rows), torch.from_numpy(gates).cuda(), bf(dout)
    dg = torch.full((T * k + pad,), 55.0, device="cuda")
    dr = r if in_place else torch.full((T * k * N + pad,), 55.0, dtype=torch.bfloat16, device="cuda")
    a = ep.ep_combine_backward_args(recv_buf=ep.ptr(r) if want_dgates else 0,
                                    gates=ep.ptr(g) if want_drows else 0, dout=ep.ptr(d),
                                    dgates=ep.ptr(dg) if want_dgates else 0,
                                    drows=ep.ptr(dr) if want_drows else 0)
    torch.cuda.synchronize()
    ep.ep_combine_backward(cfg(T, k, N), a, stream)
    torch.cuda.synchronize()
    assert (dg[T * k:] == 55).all()
    if not in_place:
        assert (dr.flatten()[T * k * N:] == 55).all()
    return (dg[:T * k].view(T, k).cpu().numpy().astype(np.float64),
            dr.flatten()[:T * k * N].view(T, k, N).float().cpu().numpy())


def check(rows, gates, dout, dgates, drows):
    N = rows.shape[2]
    r, d = rows.astype(np.float64), dout.astype(np.float64)[:, None]
    if dgates is not None:
        bound = 2.0 ** -24 * (N / 32 + 32) * np.abs(r * d).sum(-1)
        assert (np.abs(dgates - (r * d).sum(-1)) <= bound + 1e-37).all()
    if drows is not None:
        np.testing.assert_array_equal(drows, ref.bf16_round(gates[..., None] * dout[:, None]))


@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (1, 8, 7168), (3, 2, 4096), (7, 3, 24), (33, 5, 264),
                                   (2, 16, 2056), (5, 9, 1000), (300, 8, 512), (1, 33, 64),
                                   (11, 4, 16384), (700, 1, 128), (65, 6, 2048), (1, 2, 20488)])
def test_combine_backward_sizes(T, k, N):
    rows, gates, dout = inputs(T, k, N, T + N)
    dgates, drows = run(rows, gates, dout)
    check(rows, gates, dout, dgates, drows)


@pytest.mark.parametrize("T,k,N", [(4, 8, 7168), (9, 3, 72), (70, 2, 4096)])
def test_combine_backward_one_output_and_in_place(T, k, N):
    rows, gates, dout = inputs(T, k, N, 5)
    dgates, drows = run(rows, gates, dout, want_drows=False)
    check(rows, gates, dout, dgates, None)
    assert (drows == 55).all()
    dgates, drows = run(rows, gates, dout, want_dgates=False)
    check(rows, gates, dout, None, drows)
    assert (dgates == 55).all()
    check(rows, gates, dout, *run(rows, gates, dout, in_place=True))


def test_combine_backward_infinities_stay_in_their_rows():
    rows, gates, dout = inputs(4, 3, 256, 6)
    rows[1, 2, 7] = np.inf
    rows[2, 0, 3] = np.nan
    dout[3, 9] = np.inf
    gates[3, 1] = 0.0
    dgates, drows = run(rows, gates, dout)
    assert np.isinf(dgates[1, 2]) and np.isfinite(dgates[1, :2]).all()
    assert np.isnan(dgates[2, 0]) and np.isfinite(dgates[2, 1:]).all()
    assert not np.isfinite(dgates[3]).any()
    assert np.isfinite(drows[:3]).all() and np.isnan(drows[3, 1, 9]) and np.isinf(drows[3, 0, 9])
    check(rows[:1], gates[:1], dout[:1], dgates[:1], drows[:1])


def test_combine_backward_repeats_bit_for_bit_and_on_another_stream():
    rows, gates, dout = inputs(50, 8, 1024, 8)
    one = run(rows, gates, dout)
    two = run(rows, gates, dout, stream=torch.cuda.Stream())
    np.testing.assert_array_equal(one[0], two[0])
    np.testing.assert_array_equal(one[1], two[1])
    run(rows[:0], gates[:0], dout[:0])


def test_combine_backward_against_differences_of_the_combine():
    """The combine is linear in the gates and in the rows: with values on a coarse grid its
    change along a direction is what the gradient says, up to the bf16 output's rounding
    (2^-9 of outputs below 64, N = 512 of them, times |dout| <= 1)."""
    T, k, N = 6, 4, 512
    rng = np.random.default_rng(3)
    grid = lambda *s: rng.integers(-4, 5, s).astype(np.float32)
    rows, dout = grid(T, k, N), grid(T, N) / 4
    gates, step = grid(T, k) / 4, grid(T, k) / 4
    dgates, drows = run(rows, gates, dout)

    def combine(g, r):
        flags = torch.full((k + 1,), 1, dtype=torch.int64, device="cuda")
        out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        rt = torch.from_numpy(r).to("cuda", torch.bfloat16)
        gt = torch.from_numpy(g).cuda()
        a = ep.ep_combine_args(recv_buf=ep.ptr(rt), recv_count=ep.ptr(flags), gates=ep.ptr(gt),
                               out=ep.ptr(out), epoch=1, status=ep.ptr(status))
        ep.ep_combine_reduce(cfg(T, k, N), a)
        torch.cuda.synchronize()
        assert status.item() == 0
        return (out.double().cpu().numpy() * dout).sum(1)

    slack = 2 * 2.0 ** -9 * 64 * N
    diff = combine(gates + step, rows) - combine(gates, rows)
    assert (np.abs(diff - (dgates * step).sum(1)) <= slack).all()
    move = grid(T, k, N)
    diff = combine(gates, rows + move) - combine(gates, rows)
    assert (np.abs(diff - (drows.astype(np.float64) * move).sum((1, 2))) <= slack).all()
