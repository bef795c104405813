"""The norm of as many tokens as the configuration's checks let through."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from test_gpu_norm import norm_call

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 2


def test_most_tokens():
    n = 1
    assert ep.ep_add_rmsnorm_backward_sizes(ep.ep_config(1, 0, 1, 1, MOST, MOST, 64, 64, 128, ep.EP_BF16, -1, 0), n) > 0
    x = torch.ones(MOST, n, dtype=torch.bfloat16, device="cuda")
    residual = torch.full((MOST, n), 2.0, dtype=torch.bfloat16, device="cuda")
    for at in (0, 77777, MOST // 2, MOST - 7297, MOST - 1):
        x[at], residual[at] = -1, -4
    weight = torch.full((n,), 0.5, device="cuda")
    norm_call(x, residual, weight, 0.0, residual, x)  # sum over the residual, y over x
    torch.cuda.synchronize()
    for at in (0, 77777, MOST // 2, MOST - 7297, MOST - 1):
        assert (x[at] == -0.5).all() and (residual[at] == -5).all()
        x[at], residual[at] = 0.5, 3
    # (fp32: 3 / sqrt(9) and half of it are exact to within steps that bf16 does not see)
    assert x.min() == 0.5 and x.max() == 0.5 and residual.min() == 3 and residual.max() == 3
