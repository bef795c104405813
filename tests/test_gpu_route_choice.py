"""The router where its choice is hard to make: values packed within the rounding of a
score, ties across lanes and groups, few unmasked experts, every count of experts and
group shape, large biases. Bounds as in test_gpu_route."""

import numpy as np
import pytest

import operator_reference as ref
from test_gpu_route import check_backward, check_route, logits, run_backward, run_route, some_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_every_number_of_experts(score):
    for E in list(range(1, 70)) + [95, 96, 97, 127, 128, 129, 191, 200, 223, 224, 251, 255, 256]:
        k = min(E, 1 + E % 9)
        x = logits(9, E, "bf16" if E % 2 else "f32", E)
        dtype = "bf16" if E % 2 else "f32"
        bias = np.random.default_rng(E).normal(size=E).astype(np.float32) if E % 3 == 0 else None
        ids, g = run_route(x, dtype, score, k, bias, renorm=E % 4 != 0)
        check_route(x, dtype, score, k, ids, g, bias, renorm=E % 4 != 0)


@pytest.mark.parametrize("n", [2, 4, 8, 16, 32])
def test_every_group_size(n):
    for per in range(1, min(65, 256 // n + 2)):
        keep = 1 + per % n
        k = min(8, keep * per)
        x = logits(6, n * per, "f32", n * 100 + per, masked=per % 3)
        for score, bias, top in (("sigmoid", True, 2), ("softmax", False, 1), ("sigmoid", False, 2)):
            b = 0.1 * np.random.default_rng(per).normal(size=n * per).astype(np.float32) if bias else None
            ids, g = run_route(x, "f32", score, k, b, (n, keep, top))
            check_route(x, "f32", score, k, ids, g, b, (n, keep, top))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_values_within_rounding(score, groups):
    """score + bias of all experts within a few units in the last place of each other."""
    rng = np.random.default_rng(11)
    E, T = 256, 64
    x = (rng.normal(size=(T, E)) * 2).astype(np.float32)
    s = ref.scores(x[0].astype(np.float64), np.zeros(E, bool), score)
    bias = (1.0 - s + rng.integers(-3, 4, E) * 2.0 ** -23).astype(np.float32)
    x[1:32] = x[0]  # the row the bias was made for, again and again
    ids, g = run_route(x, "f32", score, 8, bias, groups)
    check_route(x, "f32", score, 8, ids, g, bias, groups)
    assert (ids[:32] == ids[0]).all() and (g[:32] == g[0]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_take_the_lowest_ids(dtype):
    """Logits of a few values only: ties inside lanes, across lanes, across groups."""
    rng = np.random.default_rng(4)
    for E, groups in ((256, (1, 1, 1)), (256, (8, 4, 1)), (160, (8, 2, 1)), (64, (4, 2, 1)), (40, (1, 1, 1)),
                      (12, (1, 1, 1))):
        x = rng.integers(-2, 3, (200, E)).astype(np.float32)
        x[100:] = rng.integers(0, 40, (100, E)) / 8.0
        for score in ("sigmoid", "softmax"):
            ids, g = run_route(x, dtype, score, 8, groups=groups)
            check_route(x, dtype, score, 8, ids, g, groups=groups)


@pytest.mark.parametrize("left", [0, 1, 3, 7, 8, 9, 31])
def test_few_unmasked_experts(left):
    rng = np.random.default_rng(left)
    for E in (64, 200, 256):
        x = np.full((20, E), -np.inf, np.float32)
        for t in range(20):
            x[t, rng.permutation(E)[:left]] = rng.normal(size=left)
        bias = rng.normal(size=E).astype(np.float32)
        for b in (None, bias):
            for groups in ((1, 1, 1), (4, 2, 2)):
                ids, g = run_route(x, "f32", "sigmoid", 8, b, groups)
                check_route(x, "f32", "sigmoid", 8, ids, g, b, groups)


def test_large_biases_and_logits():
    rng = np.random.default_rng(9)
    x = (rng.normal(size=(40, 128)) * 60).astype(np.float32)
    bias = (rng.integers(-2, 3, 128) * 50.0).astype(np.float32)
    low = ref.LOWEST["f32"]
    for score in ("sigmoid", "softmax"):
        ids, g = run_route(x, "f32", score, 6, bias)
        for t in range(40):
            l = x[t].astype(np.float64)
            v = ref.choice_values(l, l <= low, score, bias)
            top = np.sort(v)[::-1][:6]
            # the value is rounded to fp32 next to a bias of up to 100: 2^-18
            assert (v[ids[t]] >= top - 2.0 ** -17).all()
            want = ref.gates_of(l, ids[t], score, True, 1.0, low)
            np.testing.assert_allclose(g[t], want, rtol=1e-4, atol=1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_of_every_number_of_experts(score, renorm):
    for E in list(range(1, 40)) + [63, 64, 65, 127, 128, 129, 200, 255, 256, 258, 300]:
        k = min(E, 1 + E % 9)
        dtype = "bf16" if E % 2 else "f32"
        x, ids = logits(5, E, dtype, E), some_ids(5, E, k, E)
        dg = np.random.default_rng(E).normal(size=(5, k)).astype(np.float32)
        got, status = run_backward(x, ids, dg, dtype, score, renorm, 1.5)
        assert status == 0
        check_backward(got, x, ids, dg, dtype, score, renorm, 1.5)
