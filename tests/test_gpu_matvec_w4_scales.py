"""e2m1 scales as weights have them, 2 and less, which the codes take on (a scale past that sends its
step through sums of its own): sizes, columns, rows and batches with bytes up to 128 alone, and
the ends of the range in the form for few rows and in the one for many. Bounds as in
test_gpu_matvec_w4."""

import numpy as np
import pytest
import torch

import operator_reference as ref
from test_gpu_matvec_w4 import Call, activations
from test_gpu_matvec_w4_batches import batch

pytestmark = pytest.mark.gpu

FORM_ROWS = [1, 9, 24]  # announced rows an expert: each takes another form


def small_scales(E, N, K, seed, lowest=100):
    """Codes, and scale bytes lowest .. 128."""
    rng = np.random.default_rng(seed)
    packed = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    return packed, rng.integers(lowest, 129, (E, N, K // 32)).astype(np.uint8), None


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("announced", FORM_ROWS)
@pytest.mark.parametrize("N,K,counts", [
    (2, 128, [1]), (64, 256, [1, 0, 2]), (130, 384, [8]), (126, 1408, [0, 9, 0, 47]),
    (514, 2048, [31, 1, 16, 17, 32]), (1000, 640, [17, 33, 0, 70]), (4096, 512, [5]),
    (62, 96, [3, 65]), (2050, 1504, [3, 4, 2]),
])
def test_sizes(N, K, counts, announced, act):
    c = Call(activations(sum(counts), K, N), counts, small_scales(len(counts), N, K, K), "e2m1", 32, act)
    c.check(batch(c, announced).run())


@pytest.mark.parametrize("announced", FORM_ROWS)
@pytest.mark.parametrize("N,K", [(1, 64), (7, 224), (63, 320), (129, 1632), (2049, 64), (257, 14336)])
def test_odd_columns(N, K, announced):
    c = Call(activations(20, K, N), [2, 18], small_scales(2, N, K, N, 120), "e2m1", 32)
    c.check(batch(c, announced).run())


@pytest.mark.parametrize("announced", FORM_ROWS)
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 32, 33, 64, 65, 129])
def test_row_counts(rows, announced):
    c = Call(activations(rows, 1056, rows), [0, rows, 0], small_scales(3, 200, 1056, 1), "e2m1", 32,
             max_rows=200)
    c.check(batch(c, announced).run())


@pytest.mark.parametrize("announced", FORM_ROWS)
def test_long_k_is_cut_between_blocks(announced):
    c = batch(Call(activations(20, 14336, 3), [20], small_scales(1, 700, 14336, 2), "e2m1", 32), announced)
    c.check(c.run())
    first = c.bits
    c.C.fill_(55.0)
    c.run(torch.cuda.Stream())
    np.testing.assert_array_equal(first, c.bits)


@pytest.mark.parametrize("announced", FORM_ROWS)
def test_some_steps_with_large_scales(announced):
    """One scale past 2 in one weight row of one step: that step takes the other way."""
    packed, scales, _ = small_scales(1, 300, 1536, 5)
    scales[0, 200, 17] = 140
    c = batch(Call(activations(20, 1536, 5), [20], (packed, scales, None), "e2m1", 32), announced)
    c.check(c.run())


@pytest.mark.parametrize("announced", FORM_ROWS)
def test_infinities_stay_in_their_rows(announced):
    x = activations(40, 512, 4)
    x[3, 100], x[33, 511], x[8, 0] = np.inf, np.nan, -np.inf
    c = batch(Call(x, [40], small_scales(1, 100, 512, 4), "e2m1", 32), announced)
    out = c.run()
    with np.errstate(invalid="ignore"):
        y, size = c.want()
        clean = [i for i in range(40) if i not in (3, 33, 8)]
        assert np.isnan(out[33]).all()
        np.testing.assert_array_equal(np.isnan(out[[3, 8]]), np.isnan(y[[3, 8]]))
        np.testing.assert_array_equal(np.sign(out[[3, 8]]), np.sign(y[[3, 8]]))
        assert (np.abs(out - y)[clean] <= 2.0 ** -7.9 * np.abs(y[clean]) + size[clean]).all()


@pytest.mark.parametrize("announced", FORM_ROWS)
@pytest.mark.parametrize("low", [True, False])
def test_ends_of_the_scales(low, announced):
    """Rows of the smallest scales (2^-127 and 2^-126, whose products with the codes are subnormal
    bf16 numbers) and, with codes whose weights stay below 2^128, of the largest; a NaN
    scale makes its weight row's results NaN alone."""
    packed, scales, _ = small_scales(1, 40, 256, 6, 120)
    x = activations(20, 256, 5) * np.float32(2.0 ** (60 if low else -60))
    if low:
        scales[0, 0], scales[0, 1], scales[0, 2, ::2], scales[0, 2, 1::2] = 0, 1, 0, 1
        nan = []
    else:
        scales[0, 0], scales[0, 1] = 254, 253
        packed[0, :2] &= 0xBB  # magnitudes 0 .. 1.5
        scales[0, 3, 1] = 255
        nan = [3]
    c = batch(Call(x, [20], (packed, scales, None), "e2m1", 32), announced)
    out = c.run()
    y, size = c.want()
    assert np.isnan(out[:, nan]).all()
    ok = [n for n in range(40) if n not in nan]
    err = np.abs(out - y)[:, ok]
    assert (err <= 2.0 ** -7.9 * np.abs(y[:, ok]) + size[:, ok] + 1e-37).all()
    assert (np.abs(y[:, :2]) > (1e-25 if low else 1e10)).any()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("announced", FORM_ROWS)
def test_integer_scales_of_any_size_and_sign(announced, group):
    """Integer weights with scales from 2^-100 to 2^100, negative ones, zeros and infinities."""
    rng = np.random.default_rng(group)
    K, N = 512, 60
    packed = rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    scales = ref.bf16_round(rng.normal(size=(1, N, K // group)).astype(np.float32))
    scales *= np.exp2(rng.integers(-100, 101, (1, N, 1))).astype(np.float32)
    scales[0, 5], scales[0, 6, 0], scales[0, 7, 1], scales[0, 8] = 0, np.inf, np.nan, -0.0
    zeros = rng.integers(0, 16, scales.shape).astype(np.uint8)
    c = batch(Call(activations(20, K, 5), [20], (packed, scales, zeros), "int4z", group), announced)
    out = c.run()
    with np.errstate(invalid="ignore"):
        y, size = c.want()
        assert (out[:, [5, 8]] == 0).all() and np.isnan(out[:, 7]).all()
        np.testing.assert_array_equal(np.isfinite(out[:, 6]), np.isfinite(y[:, 6]))
        ok = [n for n in range(N) if n not in (6, 7)]
        assert (np.abs(out - y)[:, ok] <= 2.0 ** -7.9 * np.abs(y[:, ok]) + size[:, ok] + 1e-37).all()


@pytest.mark.parametrize("announced", FORM_ROWS)
def test_integer_scales_next_to_the_smallest(announced):
    """Scales around 2^-120 and subnormal ones. Split into two bf16 numbers, whose spacing there is
    2^-133 (2^-127 after the factor of 64 that the codes leave out), a weight under a scale below
    2^-120 may be off by half of that; with larger scales it is exact."""
    rng = np.random.default_rng(1)
    K, N = 256, 48
    packed = rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    bits = rng.integers(1, 0x0600, (1, N, K // 32)).astype(np.uint32)  # up to 2^-115
    bits[0, ::2] = rng.integers(0x0380, 0x0600, (N // 2, K // 32))     # from 2^-120 on
    scales = (bits << 16).view(np.float32)
    x = activations(20, K, 5) * np.float32(2.0 ** 60)
    c = batch(Call(x, [20], (packed, scales, None), "int4", 32), announced)
    out = c.run()
    y, size = c.want()
    lost = np.abs(x.astype(np.float64)).sum(1)[:, None] * 2.0 ** -128 * (np.arange(N) % 2)
    assert (np.abs(out - y) <= 2.0 ** -7.9 * np.abs(y) + size + 1.01 * lost).all()
