"""The fp8 layer's buffers are made while torch's current stream is busy, its calls go to another one."""

import pytest
import torch

from test_gpu_norm_layer import R, Block

pytestmark = pytest.mark.gpu


def test_nothing_lands_on_a_calls_rows():
    b = Block(12, True, seed=4)
    b.norm_and_route()
    s, stream = b.s, torch.cuda.Stream()
    b.long_way()
    torch.cuda.synchronize()
    want = [o.clone() for o in s.out]
    for r in range(R):
        s.layer_fp8[r] = s.ops[r] = None  # (their memory is used again, so that nothing waits for more)
        s.out[r].fill_(torch.nan)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for r in range(R):
        s.set_layer_fp8(r, b.q[r], b.qs[r], *b.W[r])
    for r in range(R):
        s.layer_forward_fp8(r, 2, stream)
    for r in range(R):
        s.combine(r, 2, stream=stream)
    stream.synchronize()
    with torch.cuda.stream(stream):
        seen = [{k: v.clone() for k, v in list(s.layer_fp8[r].items()) + list(s.ops[r].items())} for r in range(R)]
    stream.synchronize()
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all()
    for r in range(R):
        assert torch.equal(s.out[r], want[r])
        m = int(s.plans[r]["m_total"])
        for name, buffer in list(s.layer_fp8[r].items()) + list(s.ops[r].items()):
            if name in ("A_in", "in_scales", "G", "A", "a_scales"):
                now = buffer[:m].contiguous().view(torch.uint8)
                assert torch.equal(now, seen[r][name][:m].contiguous().view(torch.uint8)), name
