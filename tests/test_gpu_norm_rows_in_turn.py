"""The norm and its gradient where blocks take several rows: the rows under way at once, the buffers that take
turns and the rows asked for ahead, for every number of pieces a thread, in whole pieces and not, and with
more blocks than are resident."""

import pytest
import torch

from test_gpu_norm import norm_call
from test_gpu_norm import test_norm as check_norm
from test_gpu_norm import test_norm_backward as check_norm_backward

pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


def most_blocks(n, two_upto):
    """More blocks of rows of n than these are not resident at once, by the registers of a thread."""
    pieces, regs = (1, 64) if n <= 1024 else (2, 64) if n <= two_upto else (4, 128)
    threads = ((n + pieces * 8 - 1) // (pieces * 8) + 31) // 32 * 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return max(1, min(16, 65536 // regs // threads)) * sms


# (tokens, columns, gap between the rows): whole pieces of one, two and four a thread, then not whole ones
ROWS = [(3000, 1024, 0), (4000, 1032, 8), (4000, 2048, 0), (1500, 4096, 16), (400, 8200, 0), (400, 16384, 0),
        (6000, 203, 0), (3000, 1001, 3), (4000, 1111, 0), (1500, 4099, 1), (400, 8201, 0), (400, 16383, 1)]


@pytest.mark.parametrize("tokens,n,gap", ROWS)
@pytest.mark.parametrize("stream_type,weight_type", [(None, B), (B, F), (F, B)])
def test_several_rows_a_block(tokens, n, gap, stream_type, weight_type):
    assert tokens > 2 * most_blocks(n, 8192)
    check_norm(tokens, n, gap, stream_type, weight_type)


# beside a residual, a block more for each 6 (fp32: 3) rows of a resident one: two waves of them and more
@pytest.mark.parametrize("tokens,n,gap,stream_type", [(12000, 2048, 0, B), (6500, 2048, 8, F), (1500, 8200, 0, B),
                                                      (2600, 8200, 8, F), (800, 16384, 0, F), (4400, 4099, 0, B),
                                                      (1300, 8201, 3, F), (22500, 203, 0, B)])
def test_several_waves_of_blocks(tokens, n, gap, stream_type):
    rows = most_blocks(n, 8192) * (6 if stream_type is B else 3)
    assert tokens >= 1.5 * rows
    check_norm(tokens, n, gap, stream_type, F)


# (and 11111 and 16383 in fp32: rows of which one fits)
@pytest.mark.parametrize("tokens,n,gap", ROWS + [(400, 11111, 2)])
@pytest.mark.parametrize("h_type,weight_type,through", [(B, F, True), (F, B, True), (B, B, False), (F, F, False)])
def test_gradient_of_several_rows_a_block(tokens, n, gap, h_type, weight_type, through):
    assert tokens > 2 * most_blocks(n, 4096)
    check_norm_backward(tokens, n, gap, h_type, weight_type, through)


@pytest.mark.parametrize("tokens,n", [(4000, 2048), (400, 16384), (4000, 1111), (400, 16383)])
@pytest.mark.parametrize("stream_type", [B, F])
def test_over_the_inputs(tokens, n, stream_type):
    """Sum over the residual and y over x, of a row whose followers are asked for already."""
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(tokens, n, generator=gen).cuda().to(B)
    residual = torch.randn(tokens, n, generator=gen).cuda().to(stream_type)
    w = torch.randn(n, generator=gen).cuda()
    total, y = torch.zeros_like(residual), torch.zeros_like(x)
    norm_call(x, residual, w, 1e-5, total, y)
    norm_call(x, residual, w, 1e-5, residual, x)
    assert torch.equal(residual, total) and torch.equal(x, y)
