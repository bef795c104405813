"""The router and its gradient on the GPU against the 64-bit reference.

Choices: exact where the choice value is the logit itself. With a bias (or the sum of two
scores for a group) the fp32 values carry rounding: a score at most 4 ulp (expf 1, the
sum, the division), so chosen values agree with the exact top ones within 2^-21.
Gates and gradients: relative to the magnitude they are summed from, 2^-24 times
(16 + twice the largest logit difference, which the exponent's rounding scales with
+ E/16, the longest chain of a sum); a bf16 gradient adds half the spacing of bf16 numbers (7 stored bits), 2^-8."""

import ctypes

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
import operator_reference as ref

pytestmark = pytest.mark.gpu

SCORE = {"softmax": ep.EP_SCORE_SOFTMAX, "sigmoid": ep.EP_SCORE_SIGMOID}
DTYPE = {"f32": (torch.float32, ep.EP_LOGITS_F32), "bf16": (torch.bfloat16, ep.EP_LOGITS_BF16)}


def cfg(T, E, k):
    ranks = -(-E // 256)
    assert E % ranks == 0
    return ep.ep_config(n_ranks=ranks, my_rank=0, n_local_experts=E // ranks, top_k=k,
                        num_tokens=T, max_tokens_per_rank=max(T, 1), K=64, N=64, msg_bytes=128,
                        dtype=ep.EP_BF16, send_warps=-1, signal_mode=0)


def strided(x, dtype, stride):
    """x as device rows `stride` elements apart (the gaps hold NaN)."""
    T, E = x.shape
    buf = torch.full((max(T, 1), stride), float("nan"), dtype=DTYPE[dtype][0], device="cuda")
    buf[:T, :E] = torch.from_numpy(x).to("cuda", DTYPE[dtype][0])
    return buf


def run_route(x, dtype, score, k, bias=None, groups=(1, 1, 1), renorm=True, scale=1.0, stride=None,
              offset=0, gates=True, stream=None):
    T, E = x.shape
    stride = stride or E
    buf = strided(x, dtype, stride)
    if offset:  # rows that start at an odd element
        flat = torch.empty(buf.numel() + offset, dtype=buf.dtype, device="cuda")
        flat[offset:] = buf.flatten()
        buf = flat[offset:]
    ids = torch.full((max(T, 1), k), -7, dtype=torch.int32, device="cuda")
    g = torch.full((max(T, 1), k), float("nan"), device="cuda")
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    a = ep.ep_route_args(logits=ep.ptr(buf), logits_stride=0 if stride == E else stride,
                         logits_dtype=DTYPE[dtype][1], score=SCORE[score], bias=ep.ptr(b),
                         n_groups=groups[0], topk_groups=groups[1], group_top=groups[2],
                         renormalize=int(renorm), scale=scale, topk_ids=ep.ptr(ids),
                         gates=ep.ptr(g) if gates else 0)
    torch.cuda.synchronize()
    ep.ep_route(cfg(T, E, k), a, stream)
    torch.cuda.synchronize()
    return ids.cpu().numpy()[:T], g.cpu().numpy()[:T].astype(np.float64)


def logits(T, E, dtype, seed, masked=0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)).astype(np.float32) * 1.5
    if dtype == "bf16":
        x = ref.bf16_round(x)
    if masked:
        x[:, rng.permutation(E)[:masked]] = -np.inf
    return x


def rtol(x, E):
    f = x[np.isfinite(x) & (np.abs(x) < 1e30)]
    spread = f.max() - f.min() if f.size else 0
    return 2.0 ** -24 * (16 + 2 * spread + E / 16)


def check_route(x, dtype, score, k, ids, gates, bias=None, groups=(1, 1, 1), renorm=True, scale=1.0):
    low, E = ref.LOWEST[dtype], x.shape[1]
    exact_ids = bias is None and not (groups[1] < groups[0] and groups[2] == 2)
    eps = 2.0 ** -21
    for t in range(x.shape[0]):
        l = x[t].astype(np.float64)
        masked = (l <= low) | np.isnan(l)
        want = ref.chosen(l, masked, score, bias, k, *groups)
        assert len(set(ids[t])) == k and ids[t].min() >= 0 and ids[t].max() < E
        if exact_ids:
            np.testing.assert_array_equal(ids[t], want, err_msg=str(t))
        elif not np.array_equal(ids[t], want):
            member = np.ones(E, bool)
            if groups[1] < groups[0]:
                worth = ref.group_worth(l, masked, score, bias, groups[0], groups[2])
                floor = np.sort(worth)[::-1][groups[1] - 1]
                of = ids[t] // (E // groups[0])
                assert (worth[of] >= floor - 2 * eps).all(), t
                member = np.isin(np.arange(E) // (E // groups[0]), of)
            v = ref.choice_values(l, masked, score, bias)
            top = np.sort(v[member])[::-1][:k]
            assert (v[ids[t]] >= top - eps).all(), t
        g = ref.gates_of(l, ids[t], score, renorm, scale, low)
        np.testing.assert_allclose(gates[t], g, rtol=rtol(x, E), atol=1e-37, err_msg=str(t))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (37, 8, 2), (130, 60, 6),
                                   (65, 33, 32), (9, 100, 3), (40, 160, 6), (5, 384, 8),
                                   (6, 512, 32), (2, 1000, 10), (3, 2048, 8)])
def test_route_sizes(T, E, k, score, dtype):
    x = logits(T, E, dtype, T * 1000 + E)
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        ids, g = run_route(x, dtype, score, k, renorm=renorm, scale=scale)
        check_route(x, dtype, score, k, ids, g, renorm=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E,k,groups", [(256, 8, (8, 4, 2)), (256, 8, (8, 4, 1)), (60, 6, (4, 3, 2)),
                                        (160, 6, (8, 3, 1)), (72, 4, (24, 5, 2)), (96, 8, (96, 8, 2)),
                                        (24, 2, (2, 1, 2)), (256, 8, (8, 8, 2)), (512, 8, (16, 4, 2)),
                                        (240, 8, (40, 3, 2)), (64, 8, (8, 1, 2)), (1024, 8, (8, 4, 2))])
def test_route_groups_and_bias(E, k, groups, score, with_bias):
    x = logits(50, E, "f32", E + k, masked=3)
    bias = np.random.default_rng(E).normal(size=E).astype(np.float32) * 0.1 if with_bias else None
    ids, g = run_route(x, "f32", score, k, bias, groups)
    check_route(x, "f32", score, k, ids, g, bias, groups)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k,groups", [(8, 8, (1, 1, 1)), (96, 7, (1, 1, 1)), (256, 8, (8, 4, 2)),
                                        (64, 16, (4, 1, 1))])
def test_route_ties_masks_and_empty_rows(E, k, groups, dtype):
    """Rows of equal logits, signed zeros, -inf, the type's lowest value, nothing left."""
    low = np.float32(ref.LOWEST[dtype])
    x = np.zeros((9, E), np.float32)
    x[1, ::2] = -0.0
    x[2] = -np.inf
    x[3] = low
    x[4, :] = -np.inf
    x[4, E // 2] = 1.0
    x[5, : E // 2] = low
    x[6] = np.repeat(np.arange(E // 4), 4)[:E] % 3 * 0.5
    x[7, -1] = -np.inf
    x[8] = -80.0  # far below zero, but not masked
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, g = run_route(x, dtype, score, k, groups=groups, renorm=renorm)
            check_route(x, dtype, score, k, ids, g, groups=groups, renorm=renorm)
            assert (g[2] == 0).all() and (g[3] == 0).all()


def test_route_masked_experts_lose_against_a_negative_bias():
    """A masked expert stays behind one whose score plus bias is far below zero."""
    x = np.zeros((2, 16), np.float32)
    x[:, ::2] = -np.inf
    bias = np.full(16, -3.0)
    bias[0] = 5.0
    ids, g = run_route(x, "f32", "sigmoid", 8, bias)
    assert (ids == np.arange(1, 16, 2)).all()
    ids, g = run_route(x, "f32", "sigmoid", 4, bias, groups=(4, 2, 2))
    check_route(x, "f32", "sigmoid", 4, ids, g, bias, (4, 2, 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_nan_and_infinity(score):
    x = logits(5, 64, "f32", 3)
    x[0, 5] = np.nan
    x[1, 7] = np.inf
    x[2] = np.nan
    ids, g = run_route(x, "f32", score, 4)
    assert np.isnan(g[0]).all() and 5 not in ids[0] and np.isnan(g[2]).all()
    assert (ids[2] == np.arange(4)).all() and ids[1, 0] == 7
    assert np.isnan(g[1]).all() == (score == "softmax")
    check_route(x[3:], "f32", score, 4, ids[3:], g[3:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,stride,offset", [(100, 101, 1), (64, 64, 1), (256, 264, 0), (64, 96, 3),
                                             (37, 37, 0)])
def test_route_strides_and_alignment(E, stride, offset, dtype):
    x = logits(33, E, dtype, stride)
    ids, g = run_route(x, dtype, "sigmoid", 4, stride=stride, offset=offset)
    check_route(x, dtype, "sigmoid", 4, ids, g)


def test_route_without_gates_no_tokens_and_another_stream():
    x = logits(40, 64, "f32", 8)
    s = torch.cuda.Stream()
    ids, g = run_route(x, "f32", "softmax", 4, gates=False, stream=s)
    assert np.isnan(g).all()
    check_route(x, "f32", "softmax", 4, ids, run_route(x, "f32", "softmax", 4)[1])
    run_route(x[:0], "f32", "softmax", 4)


def test_route_is_repeatable_over_many_tokens():
    """Past one wave of blocks: every row equals the same rows routed alone."""
    x = logits(20000, 128, "f32", 12)
    ids, g = run_route(x, "f32", "softmax", 8)
    part, pg = run_route(x[19000:], "f32", "softmax", 8)
    np.testing.assert_array_equal(ids[19000:], part)
    np.testing.assert_array_equal(g[19000:], pg)
    check_route(x[:64], "f32", "softmax", 8, ids[:64], g[:64])


# ---------------------------------------------------------------- gradient


def run_backward(x, ids, dg, dtype, score, renorm, scale, stride=None, dstride=None, in_place=False):
    T, E = x.shape
    stride, dstride = stride or E, dstride or E
    buf = strided(x, dtype, stride)
    out = buf if in_place else torch.full((T, dstride), 77.0, dtype=DTYPE[dtype][0], device="cuda")
    i = torch.from_numpy(ids.astype(np.int32)).cuda()
    d = torch.from_numpy(dg.astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = ep.ep_route_backward_args(logits=ep.ptr(buf), logits_stride=stride,
                                  logits_dtype=DTYPE[dtype][1], score=SCORE[score],
                                  renormalize=int(renorm), scale=scale, topk_ids=ep.ptr(i),
                                  dgates=ep.ptr(d), dlogits=ep.ptr(out),
                                  dlogits_stride=stride if in_place else dstride,
                                  status=ep.ptr(status))
    ep.ep_route_backward(cfg(T, E, ids.shape[1]), a)
    torch.cuda.synchronize()
    gap = out[:, E:].float().cpu().numpy()
    if not in_place:
        assert (gap == 77).all()
    return out[:, :E].float().cpu().numpy().astype(np.float64), int(status.item())


def check_backward(got, x, ids, dg, dtype, score, renorm, scale):
    tol, half = rtol(x, x.shape[1]), 2.0 ** -8 if dtype == "bf16" else 0.0
    for t in range(x.shape[0]):
        want, size = ref.gates_backward(x[t].astype(np.float64), ids[t], dg[t].astype(np.float64),
                                        score, renorm, scale, ref.LOWEST[dtype])
        assert (np.abs(got[t] - want) <= tol * size + half * np.abs(want) * (1 + tol) + 1e-37).all(), t


def some_ids(T, E, k, seed):
    rng = np.random.default_rng(seed)
    return np.stack([rng.permutation(E)[:k] for _ in range(T)])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (37, 8, 2), (130, 60, 6),
                                   (65, 33, 32), (7, 101, 5), (5, 384, 8), (3, 2048, 8),
                                   (2, 1000, 32)])
def test_route_backward_sizes(T, E, k, renorm, score, dtype):
    x = logits(T, E, dtype, T + E, masked=1 if E > 8 else 0)
    ids = some_ids(T, E, k, E)
    dg = np.random.default_rng(T).normal(size=(T, k)).astype(np.float32)
    got, status = run_backward(x, ids, dg, dtype, score, renorm, 2.5)
    assert status == 0
    check_backward(got, x, ids, dg, dtype, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,stride,dstride,in_place", [(64, 64, 64, True), (63, 65, 70, False),
                                                       (128, 136, 132, False), (100, 103, 103, True)])
def test_route_backward_strides_and_in_place(E, stride, dstride, in_place, score, renorm):
    for dtype in ("f32", "bf16"):
        x, ids = logits(41, E, dtype, E), some_ids(41, E, 4, 5)
        dg = np.random.default_rng(9).normal(size=(41, 4)).astype(np.float32)
        got, _ = run_backward(x, ids, dg, dtype, score, renorm, 1.0, stride, dstride, in_place)
        check_backward(got, x, ids, dg, dtype, score, renorm, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_masked_rows(score, renorm):
    """Rows with nothing left, with masked chosen experts, with the type's lowest value."""
    for dtype in ("f32", "bf16"):
        x, ids = logits(6, 16, dtype, 2), some_ids(6, 16, 4, 3)
        x[0] = -np.inf
        x[1] = np.float32(ref.LOWEST[dtype])
        x[2, ids[2]] = -np.inf
        x[3, ids[3, 1]] = np.float32(ref.LOWEST[dtype])
        dg = np.random.default_rng(4).normal(size=(6, 4)).astype(np.float32)
        dg[0, 2] = np.inf  # in a masked place: counts for nothing
        dg[3, 1] = np.nan
        got, status = run_backward(x, ids, dg, dtype, score, renorm, 1.0)
        assert status == 0 and (got[:2] == 0).all()
        if score == "sigmoid" or renorm:
            assert (got[2] == 0).all()
        dg[3, 1] = 0  # the masked place again, as a number
        dg[0, 2] = 0
        check_backward(got, x, ids, dg, dtype, score, renorm, 1.0)


def test_route_backward_ids_out_of_range():
    x, ids = logits(4, 16, "f32", 2), some_ids(4, 16, 3, 3)
    dg = np.ones((4, 3), np.float32)
    ids[1, 1], ids[2, 0] = 16, -1
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got, status = run_backward(x, ids, dg, "f32", score, renorm, 1.0)
            assert status == ep.EP_STATUS_ROUTING
            keep = [0, 3]
            check_backward(got[keep], x[keep], ids[keep], dg[keep], "f32", score, renorm, 1.0)
            left = np.delete(ids[1], 1)[None]
            check_backward(got[1:2], x[1:2], left, dg[1:2, :2], "f32", score, renorm, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences_of_the_gates(score, renorm):
    """Directional differences of the forward's gates, step 2^-6: the third-order term is
    below 2^-12 of gradients of order one, a gate's rounding 2^-22 over the step 2^-16."""
    T, E, k, h = 8, 24, 4, 2.0 ** -6
    x = logits(T, E, "f32", 77) * 0.5
    ids, _ = run_route(x, "f32", score, k, renorm=renorm)
    rng = np.random.default_rng(5)
    dg = rng.normal(size=(T, k)).astype(np.float32)
    u = rng.normal(size=(T, E)).astype(np.float32)
    u /= np.linalg.norm(u, axis=1, keepdims=True)
    got, _ = run_backward(x, ids, dg, "f32", score, renorm, 1.0)

    def gates(y):
        """Gates of the same experts, whatever the order they come in."""
        i, g = run_route(y, "f32", score, E, renorm=False)
        all_g = np.empty((T, E))
        np.put_along_axis(all_g, i.astype(np.int64), g, 1)
        sel = np.take_along_axis(all_g, ids.astype(np.int64), 1)
        return sel / sel.sum(1, keepdims=True) if renorm else sel

    diff = ((gates(x + h * u) - gates(x - h * u)) / (2 * h) * dg).sum(1)
    np.testing.assert_allclose((got * u).sum(1), diff, atol=2e-3)
