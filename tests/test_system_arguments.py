"""What EpSystem's routing calls take and refuse before anything is launched: the calls go by
address, so a tensor of another type, size or stride would be read past its end or as something
else. No GPU: the library's calls are replaced by ones that keep their arguments."""

import dataclasses

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300 import system
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4

R, EL, K_TOP, T, INTER, H = 2, 3, 2, 5, 64, 128
E = R * EL


@pytest.fixture(scope="module", autouse=True)
def lib():
    ep.build()


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


# ------------------------------------------------------------------ gradients


def routed(tokens=T, dtype=torch.float32):
    s = make(tokens)
    for r in range(R):
        s.route(r, torch.zeros(tokens, E, dtype=dtype))
    return s


BF16 = dict(dtype=torch.bfloat16)


@pytest.mark.parametrize("name,kw", [
    ("dout", dict(dout=torch.ones((), **BF16).expand(T, H))),  # the gradient of out.sum()
    ("dout", dict(dout=torch.zeros(T, H))), ("dout", dict(dout=torch.zeros(T - 1, H, **BF16))),
    ("dout", dict(dout=torch.zeros(H, T, **BF16).t())),
    ("dout", dict(dout=torch.zeros(T, 2 * H, **BF16)[:, :H])),
    ("dout", dict(dout=torch.zeros(T, H, device="meta", **BF16))),
    ("dgates", dict(dgates=torch.zeros(T, K_TOP, **BF16))),
    ("dgates", dict(dgates=torch.zeros(T, K_TOP - 1))),
    ("dgates", dict(dgates=torch.zeros(K_TOP, T).t())),
    ("drows", dict(drows=torch.zeros(T, K_TOP, H))),
    ("drows", dict(drows=torch.zeros(T, H, **BF16))),
    ("drows", dict(drows=torch.zeros(T, K_TOP, H + 8, **BF16)[..., :H])),
])
def test_combine_backward_refuses(calls, name, kw):
    s = routed()
    calls.clear()
    args = dict(dout=torch.zeros(T, H, **BF16), dgates=torch.zeros(T, K_TOP))
    args.update(kw)
    with pytest.raises(ValueError, match=name):
        s.combine_backward(0, **args)
    assert not calls


def test_combine_backward_takes_either_gradient_and_the_receive_buffer(calls):
    s = routed()
    calls.clear()
    dout = torch.zeros(T, H, **BF16)
    s.combine_backward(0, dout, dgates=torch.zeros(T, K_TOP))
    s.combine_backward(0, dout, drows=torch.zeros(T, K_TOP, H, **BF16))
    s.combine_backward(0, dout, drows=torch.zeros(T * K_TOP, H, **BF16))
    s.combine_backward(1, dout, drows=s.recv[1])
    assert [name for name, _ in calls] == ["ep_combine_backward"] * 4
    assert calls[3][1].drows == s.recv[1].data_ptr()


@pytest.mark.parametrize("name,kw", [
    ("dgates", dict(dgates=torch.zeros(T, K_TOP, **BF16))),
    ("dgates", dict(dgates=torch.zeros(1, K_TOP).expand(T, K_TOP))),
    ("dgates", dict(dgates=torch.zeros(T, K_TOP + 1))),
    ("dlogits", dict(dlogits=torch.zeros(T, E, **BF16))),  # the logits are fp32
    ("dlogits", dict(dlogits=torch.zeros(1, E).expand(T, E))),
    ("dlogits", dict(dlogits=torch.zeros(E, T).t())),
    ("dlogits", dict(dlogits=torch.zeros(T, E - 1))),
    ("dlogits", dict(dlogits=torch.zeros(T, E, device="meta"))),
])
def test_route_backward_refuses(calls, name, kw):
    s = routed()
    calls.clear()
    args = dict(dgates=torch.zeros(T, K_TOP), dlogits=torch.zeros(T, E))
    args.update(kw)
    with pytest.raises(ValueError, match=name):
        s.route_backward(0, **args)
    assert not calls


def test_route_backward_takes_rows_any_stride_apart(calls):
    s = routed(dtype=torch.bfloat16)
    wide = torch.zeros(T, E + 2, **BF16)
    s.route_backward(1, torch.zeros(T, K_TOP), wide[:, 1:E + 1])
    assert calls[-1][1].dlogits == wide.data_ptr() + 2 and calls[-1][1].dlogits_stride == E + 2
    one = routed(1)
    one.route_backward(0, torch.zeros(1, K_TOP), torch.zeros(E, 1).t())
    assert calls[-1][1].dlogits_stride == 0


# -------------------------------------------------------------- 4-bit weights


def w4_layer(fmt=ep.EP_W4_INT, group=32, zeros=True):
    gen = torch.Generator().manual_seed(0)
    return (torch.zeros(T, H, **BF16),
            quantize_w4(torch.randn(EL, 2 * INTER, H, generator=gen), fmt, group, zeros),
            quantize_w4(torch.randn(EL, H, INTER, generator=gen), fmt, group, zeros))


@pytest.mark.parametrize("fmt,group,zeros", [(ep.EP_W4_INT, 32, True), (ep.EP_W4_INT, 64, False),
                                             (ep.EP_W4_E2M1, 32, False)])
def test_layer_takes_quantized_weights(fmt, group, zeros):
    make().set_layer_w4(0, *w4_layer(fmt, group, zeros))


def test_layer_refuses_what_the_products_would_read_past():
    X, W1, W2 = w4_layer()
    change = dataclasses.replace
    strided = torch.empty(EL, INTER // 2, H, dtype=torch.uint8).transpose(1, 2)
    assert strided.shape == W2.codes.shape
    for bad in [
        (X.float(), W1, W2), (torch.zeros(T, 2 * H, **BF16)[:, :H], W1, W2),
        (torch.zeros(1, H, **BF16).expand(T, H), W1, W2),
        (X, W2, W1),                                             # the two exchanged
        (X, change(W1, codes=W1.codes[:EL - 1]), W2),            # an expert short
        (X, change(W1, scales=W1.scales[..., :1]), W2),
        (X, change(W1, group_size=64), W2),                      # scales of groups of 32
        (X, change(W1, scales=W1.scales.float()), W2),
        (X, W1, change(W2, codes=strided)),
        (X, W1, change(W2, zeros=W2.zeros[:, :1])),
        (X, W1, change(W2, w_format=ep.EP_W4_E2M1)),             # bf16 scales
        (X, W1, change(W2, w_format=2)), (X, W1, change(W2, group_size=48)),
        (X, W1, change(W2, group_size=0)),
        (X, W1, change(W2, codes=W2.codes.to("meta"))),
    ]:
        s = make()
        with pytest.raises(ValueError):
            s.set_layer_w4(0, *bad)
        assert s.layer_w4[0] is None
