"""The 4-bit products with batch sizes that make a pass over the weights serve 16 and 64
rows (the choice goes by the configuration's tokens), against the same 64-bit reference
and bounds as the single-token form; ranges of rows below, at and past a pass."""

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
from test_gpu_matvec_w4 import FORMATS, Call, activations, weights

pytestmark = pytest.mark.gpu


def batch(c, rows):
    """Let the configuration announce `rows` rows for every expert."""
    c.cfg.num_tokens = c.cfg.max_tokens_per_rank = rows * c.E
    c.args.max_rows = max(c.args.max_rows, 1)
    return c


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("rows", [9, 17, 24])
@pytest.mark.parametrize("N,K,counts", [
    (130, 384, [20, 33]), (126, 1408, [0, 9, 0, 47]), (514, 2048, [31, 1, 16, 17, 32]),
    (1000, 640, [17, 33, 0, 70]),
])
def test_w4_batches(N, K, counts, rows, fmt, group):
    for act in (False, True):
        c = Call(activations(sum(counts), K, N), counts, weights(len(counts), N, K, fmt, group, K),
                 fmt, group, act)
        c.check(batch(c, rows).run())


@pytest.mark.parametrize("announced", [9, 17, 24])
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 24, 31, 32, 33, 64, 65, 129])
def test_w4_batch_row_counts(rows, announced):
    for fmt, group in (("int4z", 64), ("e2m1", 32)):
        c = Call(activations(rows, 1056 if group == 32 else 1088, rows), [rows, 0, rows * 0],
                 weights(3, 200, 1056 if group == 32 else 1088, fmt, group, 1), fmt, group,
                 max_rows=200)
        c.check(batch(c, announced).run())


@pytest.mark.parametrize("announced", [1, 9, 17, 24])
def test_w4_many_steps_for_every_block(announced):
    """Rings that turn many times, tiles cut between blocks and whole ones, repeated."""
    counts = [40, 3, 0, 28, 17, 32, 5, 9]
    for fmt, group in (("e2m1", 32), ("int4", 128)):
        c = batch(Call(activations(sum(counts), 4096, 1), counts,
                       weights(8, 3000, 4096, fmt, group, 2), fmt, group), announced)
        c.check(c.run())
        first = c.bits
        for stream in (torch.cuda.Stream(), None):
            c.C.fill_(55.0)
            c.run(stream)
            np.testing.assert_array_equal(first, c.bits)


@pytest.mark.parametrize("announced", [9, 17, 24])
def test_w4_batches_keep_infinities_in_their_rows(announced):
    x = activations(40, 512, 4)
    x[3, 100], x[33, 511], x[8, 0] = np.inf, np.nan, -np.inf
    c = batch(Call(x, [40], weights(1, 100, 512, "int4z", 64, 4), "int4z", 64), announced)
    out = c.run()
    with np.errstate(invalid="ignore"):
        y, size = c.want()
        clean = [i for i in range(40) if i not in (3, 33, 8)]
        assert np.isnan(out[33]).all()
        np.testing.assert_array_equal(np.isnan(out[[3, 8]]), np.isnan(y[[3, 8]]))
        assert (np.abs(out - y)[clean] <= 2.0 ** -7.9 * np.abs(y[clean]) + size[clean]).all()


@pytest.mark.parametrize("announced", [9, 17, 24])
def test_w4_batches_skip_bad_gather_indices(announced):
    T, K, N = 20, 320, 72
    c = batch(Call(activations(T, K, 8), [T], weights(1, N, K, "int4z", 32, 9), "int4z", 32),
              max(T, announced))
    want = c.run()
    x = torch.zeros(c.cfg.num_tokens, K, dtype=torch.bfloat16, device="cuda")
    x[:T] = c.A
    gi = torch.arange(T, dtype=torch.int32, device="cuda")
    gi[5], gi[18] = -3, c.cfg.num_tokens
    c.args.A, c.args.gather_idx, c.args.x_ptrs[0] = 0, ep.ptr(gi), ep.ptr(x)
    c.C.fill_(55.0)
    out = c.run()
    assert c.status.item() == ep.EP_STATUS_BOUNDS
    keep = [i for i in range(T) if i not in (5, 18)]
    np.testing.assert_array_equal(out[keep], want[keep])
    assert (out[[5, 18]] == 55).all()
