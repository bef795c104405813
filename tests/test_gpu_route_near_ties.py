"""Groups of experts whose worths, sums of two values with large biases of opposite sign,
lie within the rounding next to those biases of each other.

The same experts are routed twice: in eight groups, which a warp takes in registers by
approximate values, and with a ninth group of masked experts behind them, which the form that
computes every value exactly takes. Both evaluate 1 / (1 + e^-l) + bias in fp32 alike, so they
have to choose alike, expert by expert. Against 64 bits a value next to a bias of up to 128 carries
two roundings (the score's, below 2^-21, and the sum's, 2^-18), a worth two values, the difference
of two worths four: 2^-16 + 2^-19."""

import numpy as np
import pytest

import operator_reference as ref
from test_gpu_route import rtol, run_route

pytestmark = pytest.mark.gpu

N, PER, KEEP = 8, 8, 4


def near_tied(T, large, seed, pair):
    """Logits whose groups differ by a few units in the last place of the scores, and biases
    that make every group worth (score + large) + (score - large). ``pair``: all groups far
    apart but two, of which one is kept: the lower one where they are equal after rounding."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, N, PER)).astype(np.float32)
    off = rng.normal(size=(T, N)) * 4e-6
    x[:, :, 0] = (rng.normal(size=(T, 1)) * (1 + off)).astype(np.float32)
    x[:, :, 1] = rng.normal(size=(T, 1)).astype(np.float32)
    if pair:
        x[:, :KEEP - 1, 0] = [7, 6, 5]
        x[:, KEEP + 1:, 0] = [-5, -6, -7]
    bias = np.full((N, PER), -2000, np.float32)
    bias[:, 0], bias[:, 1] = large, -large
    return x.reshape(T, -1), bias.reshape(-1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pair", [True, False])
@pytest.mark.parametrize("large", [3.0, 100.0, 1000.0])
def test_group_sums_next_to_large_biases(large, pair, dtype):
    T = 20000
    x, bias = near_tied(T, large, int(large), pair)
    if dtype == "bf16":
        x = ref.bf16_round(x)
    ids, g = run_route(x, dtype, "sigmoid", 8, bias, (N, KEEP, 2))
    more = np.concatenate((x, np.full((T, PER), -np.inf, np.float32)), 1)
    want, wg = run_route(more, dtype, "sigmoid", 8, np.append(bias, np.zeros(PER)), (N + 1, KEEP, 2))
    wrong = (ids != want).any(1).sum()
    assert wrong == 0, f"{wrong} of {T} tokens"
    np.testing.assert_allclose(g, wg, rtol=2 * rtol(x, N * PER))  # (sums in another order)


def test_group_sums_against_64_bits():
    x, bias = near_tied(500, 100.0, 7, False)
    x[:250, ::PER] = np.random.default_rng(3).normal(size=(250, N))  # some that are far apart
    ids, _ = run_route(x, "f32", "sigmoid", 8, bias, (N, KEEP, 2))
    for t in range(len(x)):
        l = x[t].astype(np.float64)
        worth = ref.group_worth(l, np.zeros(l.size, bool), "sigmoid", bias, N, 2)
        kept = set(ids[t] // PER)
        rest = [worth[g] for g in range(N) if g not in kept]
        assert min(worth[g] for g in kept) >= np.sort(worth)[::-1][KEEP - 1] - 2.0 ** -16 - 2.0 ** -19
        assert len(kept) <= KEEP and rest


def test_one_disabled_expert_in_every_group():
    """A bias of -1e9 on one expert of each group takes that expert out and decides nothing else."""
    rng = np.random.default_rng(12)
    x = rng.normal(size=(300, N * 4)).astype(np.float32)
    bias = (0.1 * rng.normal(size=N * 4)).astype(np.float32)
    bias[::4] = -1e9
    ids, g = run_route(x, "f32", "sigmoid", 6, bias, (N, KEEP, 2))
    keep = np.arange(N * 4) % 4 != 0
    new_id = np.cumsum(keep) - 1
    few, fg = run_route(np.ascontiguousarray(x[:, keep]), "f32", "sigmoid", 6, bias[keep], (N, KEEP, 2))
    np.testing.assert_array_equal(new_id[ids], few)
    np.testing.assert_allclose(g, fg, rtol=2.0 ** -20)
