"""+inf among the logits: under the softmax every gate of the token is NaN, whichever experts the
biases make it choose; the sigmoid of +inf is 1 and its gates stay numbers."""

import numpy as np
import pytest

import operator_reference as ref
from test_gpu_route import check_route, logits, run_route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,groups", [(8, (1, 1, 1)), (13, (1, 1, 1)), (64, (1, 1, 1)), (256, (8, 4, 2)),
                                      (96, (4, 2, 1)), (72, (9, 3, 2)), (384, (1, 1, 1))])
def test_infinite_logit(E, groups, renorm, with_bias, dtype):
    k = 4
    x = logits(12, E, dtype, E)
    for t in range(8):  # the last tokens have none
        x[t, (E - 1) * t // 7] = np.inf
    x[3, 1] = np.inf  # two of them
    bias = np.random.default_rng(E).normal(size=E).astype(np.float32) if with_bias else None
    ids, g = run_route(x, dtype, "softmax", k, bias, groups, renorm)
    assert np.isnan(g[:8]).all()
    for t in range(8):
        assert len(set(ids[t])) == k and ids[t].min() >= 0 and ids[t].max() < E
    check_route(x[8:], dtype, "softmax", k, ids[8:], g[8:], bias, groups, renorm)
    ids, g = run_route(x, dtype, "sigmoid", k, bias, groups, renorm)
    check_route(x, dtype, "sigmoid", k, ids, g, bias, groups, renorm)
    assert np.isfinite(g).all()


def test_infinite_logit_that_the_bias_keeps_out():
    """The expert with the infinite logit is not chosen: the gates are NaN all the same."""
    for E in (8, 40, 300):
        x = np.zeros((1, E), np.float32)
        x[0, E - 1] = np.inf
        bias = np.zeros(E)
        bias[E - 1] = -5
        ids, g = run_route(x, "f32", "softmax", 3, bias)
        assert np.isnan(g).all()
        assert np.isnan(ref.gates_of(x[0].astype(float), ids[0], "softmax", True, 1.0, ref.LOWEST["f32"])).all()
