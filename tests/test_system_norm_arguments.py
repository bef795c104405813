"""What EpSystem's norm, fp8 layer and layer of a few tokens take and refuse before anything is
launched. No GPU: the library's calls are replaced by ones that keep their arguments."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300 import system
from moe_expert_gemm_gb300.system import EpSystem

R, EL, K_TOP, T, INTER, H = 2, 3, 2, 5, 128, 512
B = dict(dtype=torch.bfloat16)
Q = dict(dtype=torch.float8_e4m3fn)


@pytest.fixture(scope="module", autouse=True)
def lib():
    ep.build()


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("ep_add_rmsnorm", "ep_add_rmsnorm_backward", "ep_layer_few", "ep_swiglu_e4m3", "ep_plan",
                 "ep_dispatch_gather", "grouped_gemm_combine_send"):
        monkeypatch.setattr(system, name, lambda cfg, a, *rest, name=name: seen.append((name, cfg, a)))
    return seen


def make(dtype="bf16", tokens=T, n=H):
    return EpSystem(R, EL, K_TOP, tokens, K=INTER, N=n, device="cpu", max_tokens=max(tokens, 1), dtype=dtype)


X, W = torch.zeros(T, H, **B), torch.zeros(H)


@pytest.mark.parametrize("name,kw", [
    ("x", dict(x=torch.zeros(T, H))), ("x", dict(x=torch.zeros(T - 1, H, **B))),
    ("x", dict(x=torch.zeros(1, H, **B).expand(T, H))), ("x", dict(x=torch.zeros(H, T, **B).t())),
    ("x", dict(x=torch.zeros(T, H, device="meta", **B))), ("x", dict(x=torch.zeros(T, 2 * H, **B)[:, ::2])),
    ("weight", dict(weight=torch.zeros(H - 1))), ("weight", dict(weight=torch.zeros(2 * H)[::2])),
    ("weight", dict(weight=torch.zeros(H, dtype=torch.float16))),
    ("residual", dict(residual=torch.zeros(T, H, dtype=torch.float16))),
    ("residual", dict(residual=torch.zeros(T, H + 1))),
    ("sum", dict(residual=torch.zeros(T, H), sum=torch.zeros(T, H, **B))),
    ("sum", dict(sum=torch.zeros(T, H - 1))), ("sum", dict(sum=torch.zeros(1, H).expand(T, H))),
    ("y", dict(y=torch.zeros(T, H))), ("y", dict(y=torch.zeros(T + 1, H, **B))),
    ("q", dict(q=torch.zeros(T, H, dtype=torch.float8_e5m2))), ("q", dict(q=torch.zeros(T, 2 * H, **Q)[:, :H])),
    ("q_scales", dict(q=torch.zeros(T, H, **Q), q_scales=torch.zeros(T, H // 128 + 1))),
    ("q_scales", dict(q=torch.zeros(T, H, **Q), q_scales=torch.zeros(T, H // 128, **B))),
])
def test_norm_refuses(calls, name, kw):
    args = dict(x=X, weight=W, y=torch.zeros(T, H, **B))
    args.update(kw)
    with pytest.raises(ValueError, match=name):
        make().add_rmsnorm(0, **args)
    assert not calls


def test_norm_passes_types_and_strides(calls):
    wide, res = torch.zeros(T, 2 * H, **B)[:, :H], torch.zeros(T, H + 4)[:, 4:]
    q, s = torch.zeros(T, H, dtype=torch.uint8), torch.zeros(T, H // 128)
    make().add_rmsnorm(1, wide, W.bfloat16(), residual=res, sum=res, y=wide, q=q, q_scales=s, eps=1e-3)
    (name, cfg, a), = calls
    assert cfg.my_rank == 1 and a.hidden == H and abs(a.eps - 1e-3) < 1e-9
    assert a.x == a.y == wide.data_ptr() and a.x_stride == a.y_stride == 2 * H
    assert a.residual == a.sum == res.data_ptr() and a.residual_stride == a.sum_stride == H + 4
    assert a.residual_dtype == ep.EP_ROWS_F32 and a.weight_dtype == ep.EP_ROWS_BF16
    assert a.q == q.data_ptr() and a.q_scales == s.data_ptr()


@pytest.mark.parametrize("name,kw", [
    ("h", dict(h=torch.zeros(T, H, dtype=torch.float16))), ("h", dict(h=torch.zeros(T, H - 1))),
    ("dy", dict(dy=torch.zeros(T, H))), ("dy", dict(dy=torch.ones((), **B).expand(T, H))),
    ("dsum", dict(dsum=torch.zeros(T, H, **B))), ("dh", dict(dh=torch.zeros(T, H, **B))),
    ("dx", dict(dx=torch.zeros(T, H))), ("dweight", dict(dweight=torch.zeros(H, **B))),
    ("dweight", dict(dweight=torch.zeros(2 * H)[::2])), ("weight", dict(weight=torch.zeros(H + 1))),
])
def test_norm_backward_refuses(calls, name, kw):
    args = dict(h=torch.zeros(T, H), dy=X, weight=W, dh=torch.zeros(T, H))
    args.update(kw)
    with pytest.raises(ValueError, match=name):
        make().add_rmsnorm_backward(0, **args)
    assert not calls


def test_norm_backward_brings_a_workspace(calls):
    h = torch.zeros(T, H, **B)
    make().add_rmsnorm_backward(0, h, X, W, dh=h, dweight=torch.zeros(H))
    make().add_rmsnorm_backward(0, h, X, W, dsum=h, dx=X)
    (_, _, a), (_, _, b) = calls
    assert a.workspace and a.workspace_bytes >= T * H * 4 and a.h_dtype == ep.EP_ROWS_BF16
    assert not b.workspace and not b.dweight and b.dsum == h.data_ptr() and b.dx == X.data_ptr()


def few(dtype="bf16"):
    s = make(dtype)
    s.set_routing(torch.zeros(R, T, K_TOP, dtype=torch.int32).numpy())
    for r in range(R):
        s.set_gates(r, torch.zeros(T, K_TOP).numpy())
    if dtype == "bf16":
        s.set_layer_few(0, torch.zeros(EL, 2 * INTER, H, **B), torch.zeros(EL, H, INTER, **B))
    else:
        s.set_layer_few(0, torch.zeros(EL, 2 * INTER, H, **Q), torch.zeros(EL, H, INTER, **Q),
                        torch.zeros(EL, 2 * INTER // 128, H // 128), torch.zeros(EL, H // 128, INTER // 128))
    return s


@pytest.mark.parametrize("name,W1,W2", [
    ("W1", torch.zeros(EL, INTER, H, **B), torch.zeros(EL, H, INTER, **B)),
    ("W1", torch.zeros(EL, 2 * INTER, H), torch.zeros(EL, H, INTER, **B)),
    ("W2", torch.zeros(EL, 2 * INTER, H, **B), torch.zeros(EL, INTER, H, **B).transpose(1, 2)),
    ("W2", torch.zeros(EL, 2 * INTER, H, **B), torch.zeros(EL - 1, H, INTER, **B)),
])
def test_few_refuses_weights(name, W1, W2):
    with pytest.raises(ValueError, match=name):
        make().set_layer_few(0, W1, W2)


def test_few_refuses_fp8_weights():
    W1, W2 = torch.zeros(EL, 2 * INTER, H, **Q), torch.zeros(EL, H, INTER, **Q)
    s1, s2 = torch.zeros(EL, 2 * INTER // 128, H // 128), torch.zeros(EL, H // 128, INTER // 128)
    s = make("fp8_1d2d")
    for args in ((W1, W2), (W1, W2, s1), (W1, W2, s1[:, :1], s2), (W1, W2, s1, s2.bfloat16()),
                 (W1.view(torch.int8), W2, s1, s2)):
        with pytest.raises(ValueError):
            s.set_layer_few(0, *args)
    s.set_layer_few(0, W1.view(torch.uint8), W2, s1, s2)


@pytest.mark.parametrize("dtype,name,kw", [
    ("bf16", "x", dict(x=torch.zeros(T, H))), ("bf16", "x", dict(x=torch.zeros(T, 2 * H, **B)[:, :H])),
    ("bf16", "out", dict(out=torch.zeros(T, H))), ("bf16", "out", dict(out=torch.zeros(T - 1, H, **B))),
    ("fp8_1d2d", "x", dict(x=X)), ("fp8_1d2d", "scales", dict(x_scales=None)),
    ("fp8_1d2d", "x_scales", dict(x_scales=torch.zeros(T, H // 64))),
])
def test_few_refuses_tokens(calls, dtype, name, kw):
    s = few(dtype)
    args = dict(x=X, out=torch.zeros(T, H, **B))
    if dtype != "bf16":
        args.update(x=torch.zeros(T, H, **Q), x_scales=torch.zeros(T, H // 128))
    args.update(kw)
    with pytest.raises(ValueError, match=name):
        s.layer_few(0, **args)
    assert not calls


def test_few_takes_another_ranks_tokens(calls):
    s = few()
    out = torch.zeros(T, H, **B)
    s.layer_few(0, X, out)
    s.layer_few(0, X, out, source=1)
    (_, c, a), (_, _, b) = calls
    assert c.my_rank == 0 and a.topk_ids == s.topk[0].data_ptr() and b.topk_ids == s.topk[1].data_ptr()
    assert a.gates == s.gates[0].data_ptr() and b.gates == s.gates[1].data_ptr()
    assert a.workspace_bytes == ep.ep_layer_few_sizes(c)


def fp8_layer(s):
    return (torch.zeros(T, H, **Q), torch.zeros(T, H // 128), torch.zeros(EL, 2 * INTER, H, **Q),
            torch.zeros(EL, 2 * INTER // 128, H // 128), torch.zeros(EL, H, INTER, **Q),
            torch.zeros(EL, H // 128, INTER // 128))


def test_fp8_layer(calls):
    s = make("fp8_1d2d")
    s.topk = s._route_ids
    for r in range(R):
        s.plan(r)
        s.set_layer_fp8(r, *fp8_layer(s))
    calls.clear()
    s.layer_forward_fp8(1, epoch=3)
    names = [n for n, _, _ in calls]
    assert names == ["ep_dispatch_gather"] * 2 + ["grouped_gemm_combine_send", "ep_swiglu_e4m3",
                                                  "grouped_gemm_combine_send"]
    codes, scales, up, act, down = (a for _, _, a in calls)
    assert codes.hidden * 2 == H and scales.hidden * 2 == H // 128 * 4
    assert calls[2][1].dtype == ep.EP_FP8_1D2D and (calls[2][1].K, calls[2][1].N) == (H, 2 * INTER)
    assert up.A == codes.A_in and up.a_scales == scales.A_in and up.p3_control == -1
    assert act.G == up.C and (down.A, down.a_scales) == (act.q, act.q_scales)


@pytest.mark.parametrize("i", range(6))
def test_fp8_layer_refuses(i):
    s = make("fp8_1d2d")
    s.topk = s._route_ids
    s.plans[0] = dict(capacity=10)
    ops = list(fp8_layer(s))
    ops[i] = ops[i][..., :-1]
    with pytest.raises(ValueError):
        s.set_layer_fp8(0, *ops)


def test_fp8_layer_refuses_sizes():
    for s in (make("bf16"), make("fp8_1d2d", n=384)):
        with pytest.raises(ValueError, match="fp8 layer"):
            s.set_layer_fp8(0, *fp8_layer(s))
