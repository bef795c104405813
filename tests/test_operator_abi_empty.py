"""The router, its gradient and the combine's gradient for no tokens at all: no tensor has an
address then, and nothing is launched (no GPU)."""

import ctypes

import pytest

import moe_expert_gemm_gb300 as ep


@pytest.fixture(scope="module", autouse=True)
def lib():
    ep.build()


@pytest.mark.parametrize("name,args", [("ep_route", ep.ep_route_args(scale=1.0)),
                                       ("ep_route_backward", ep.ep_route_backward_args(scale=1.0)),
                                       ("ep_combine_backward", ep.ep_combine_backward_args())])
def test_no_tokens_need_no_addresses(name, args):
    conf = ep.ep_config(n_ranks=2, my_rank=0, n_local_experts=8, top_k=4, num_tokens=0,
                        max_tokens_per_rank=32, K=256, N=128, msg_bytes=256, dtype=ep.EP_BF16,
                        send_warps=-1, signal_mode=0)
    assert ep.raw_call(name, ctypes.byref(conf), ctypes.byref(args), None) == ep.EP_OK
    conf.num_tokens = 1
    assert ep.raw_call(name, ctypes.byref(conf), ctypes.byref(args), None) == ep.EP_ERR_INVALID_ARG
