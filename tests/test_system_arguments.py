"""What EpSystem's routing calls take and refuse before anything is launched: the calls go by
address, so a tensor of another type, size or stride would be read past its end or as something
else. No GPU: the library's calls are replaced by ones that keep their arguments."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300 import system
from moe_expert_gemm_gb300.system import EpSystem

R, EL, K_TOP, T, INTER, H = 2, 3, 2, 5, 64, 128
E = R * EL


@pytest.fixture
def calls(monkeypatch):
    """Every call's (name, arguments), nothing launched."""
    seen = []
    for name in ("ep_route", "ep_route_backward", "ep_combine_backward", "ep_matvec_w4",
                 "ep_scatter_send", "ep_plan"):
        monkeypatch.setattr(system, name, lambda cfg, a, *rest, name=name: seen.append((name, a)))
    return seen


def make(tokens=T, **kw):
    return EpSystem(R, EL, K_TOP, tokens, K=INTER, N=H, device="cpu", max_tokens=max(tokens, 1), **kw)


@pytest.mark.parametrize("what,logits", [
    ("one row for all tokens", torch.zeros(1, E).expand(T, E)),
    ("overlapping rows", torch.zeros(100).as_strided((T, E), (E - 1, 1))),
    ("a transposed view", torch.zeros(E, T).t()),
    ("every other column", torch.zeros(T, 2 * E)[:, ::2]),
    ("too few tokens", torch.zeros(T - 1, E)),
    ("too few experts", torch.zeros(T, E - 1)),
    ("another type", torch.zeros(T, E, dtype=torch.float16)),
    ("64 bits", torch.zeros(T, E, dtype=torch.float64)),
    ("another device", torch.zeros(T, E, device="meta")),
])
def test_route_refuses_logits(calls, what, logits):
    with pytest.raises(ValueError, match="logits"):
        make().route(0, logits)
    assert not calls


@pytest.mark.parametrize("bias", [
    torch.zeros(E, dtype=torch.bfloat16), torch.zeros(E - 1), torch.zeros(E + 1),
    torch.zeros(1).expand(E), torch.zeros(2 * E)[::2], torch.zeros(E, device="meta"),
])
def test_route_refuses_bias(calls, bias):
    with pytest.raises(ValueError, match="bias"):
        make().route(0, torch.zeros(T, E), bias=bias)
    assert not calls


@pytest.mark.parametrize("logits,stride", [
    (torch.zeros(T, E), E), (torch.zeros(T, E + 3)[:, 1:E + 1], E + 3),
    (torch.zeros(T, E, dtype=torch.bfloat16), E), (torch.zeros(3 * T, E)[::3], 3 * E),
])
def test_route_takes_rows_any_stride_apart(calls, logits, stride):
    s = make()
    s.route(1, logits, bias=torch.zeros(E))
    (name, a), = calls
    assert name == "ep_route" and a.logits == logits.data_ptr() and a.logits_stride == stride
    assert a.logits_dtype == (ep.EP_LOGITS_F32 if logits.dtype == torch.float32 else ep.EP_LOGITS_BF16)


@pytest.mark.parametrize("logits", [
    torch.zeros(E, 1).t(),            # one token: strides (1, 1)
    torch.zeros(E).expand(1, E),
    torch.zeros(1, 4 * E)[:, :E],
])
def test_route_of_one_token_needs_no_row_stride(calls, logits):
    make(1).route(0, logits)
    assert calls[0][1].logits_stride == 0  # back to back


def test_route_of_no_tokens(calls):
    make(0).route(0, torch.zeros(0, E))
    assert len(calls) == 1
