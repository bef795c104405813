"""Arguments of the router, its gradient, the combine's gradient and the 4-bit products:
layouts against the header, refusals before any launch (no GPU)."""

import ctypes
import os
import subprocess

import pytest

import moe_expert_gemm_gb300 as ep

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x1000000  # an aligned address that no refused call touches
BAD, UNSUP = ep.EP_ERR_INVALID_ARG, ep.EP_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    ep.build()
    return ep.load()


def cfg(**kw):
    base = dict(n_ranks=2, my_rank=0, n_local_experts=8, top_k=4, num_tokens=32,
                max_tokens_per_rank=32, K=256, N=128, dtype=ep.EP_BF16, send_warps=-1,
                signal_mode=0)
    base.update(kw)
    return ep.ep_config(msg_bytes=2 * base["N"], **base)


def call(name, c, a):
    return ep.raw_call(name, ctypes.byref(c) if c is not None else None,
                       ctypes.byref(a) if a is not None else None, None)


def route_args(**kw):
    base = dict(logits=P, logits_dtype=ep.EP_LOGITS_F32, score=ep.EP_SCORE_SIGMOID, bias=P,
                n_groups=4, topk_groups=2, group_top=2, scale=1.0, topk_ids=P, gates=P)
    base.update(kw)
    return ep.ep_route_args(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=0), BAD), (dict(topk_ids=0), BAD), (dict(logits=P + 2), BAD),
    (dict(logits_dtype=2), BAD), (dict(score=2), BAD), (dict(n_groups=3), BAD),
    (dict(n_groups=-1), BAD), (dict(topk_groups=5), BAD), (dict(topk_groups=0), BAD),
    (dict(group_top=3), BAD), (dict(n_groups=8, topk_groups=1), BAD),
    (dict(logits_stride=15), BAD), (dict(logits_stride=-16), BAD),
    (dict(bias=P + 1), BAD), (dict(gates=P + 2), BAD), (dict(topk_ids=P + 2), BAD),
])
def test_route_refusals(kw, code):
    assert call("ep_route", cfg(), route_args(**kw)) == code


def test_route_limits():
    c = cfg(n_local_experts=64, top_k=33)
    assert call("ep_route", c, route_args(n_groups=1)) == UNSUP
    assert call("ep_route", cfg(), None) == BAD
    assert call("ep_route", None, route_args()) == BAD
    assert call("ep_route", cfg(num_tokens=0), route_args(logits=0, topk_ids=0)) == ep.EP_OK


def back_args(**kw):
    base = dict(logits=P, logits_dtype=ep.EP_LOGITS_BF16, score=ep.EP_SCORE_SOFTMAX, scale=1.0,
                topk_ids=P, dgates=P, dlogits=P, status=P)
    base.update(kw)
    return ep.ep_route_backward_args(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=0), BAD), (dict(topk_ids=0), BAD), (dict(dgates=0), BAD), (dict(dlogits=0), BAD),
    (dict(status=0), BAD), (dict(dlogits=P + 1), BAD), (dict(dlogits_stride=8), BAD),
    (dict(logits_dtype=-1), BAD), (dict(score=-1), BAD), (dict(logits_stride=1), BAD),
])
def test_route_backward_refusals(kw, code):
    assert call("ep_route_backward", cfg(), back_args(**kw)) == code


def test_route_backward_limits():
    assert call("ep_route_backward", cfg(n_local_experts=64, top_k=33), back_args()) == UNSUP
    assert call("ep_route_backward", cfg(num_tokens=0), back_args(logits=0)) == ep.EP_OK


@pytest.mark.parametrize("kw", [
    dict(dgates=0, drows=0), dict(dout=0), dict(recv_buf=0), dict(gates=0), dict(dout=P + 8),
    dict(recv_buf=P + 8), dict(drows=P + 8), dict(dgates=P + 2), dict(gates=P + 2),
])
def test_combine_backward_refusals(kw):
    base = dict(recv_buf=P, gates=P, dout=P, dgates=P, drows=P)
    base.update(kw)
    a = ep.ep_combine_backward_args(**base)
    assert call("ep_combine_backward", cfg(), a) == BAD


def test_combine_backward_needs_whole_vectors():
    a = ep.ep_combine_backward_args(recv_buf=P, gates=P, dout=P, dgates=P, drows=P)
    assert call("ep_combine_backward", cfg(N=132), a) == BAD
    assert call("ep_combine_backward", cfg(num_tokens=0), a) == ep.EP_OK


def w4_args(**kw):
    base = dict(A=P, W=P, w_scales=P, w_format=ep.EP_W4_INT, group_size=64, expert_offsets=P,
                max_rows=64, local_activation=ep.EP_ACT_NONE, C=P, workspace=P,
                workspace_bytes=1 << 40, status=P)
    base.update(kw)
    return ep.ep_w4_args(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(A=0), BAD), (dict(A=P + 8), BAD), (dict(W=0), BAD), (dict(W=P + 4), BAD),
    (dict(w_scales=0), BAD), (dict(w_scales=P + 1), BAD), (dict(C=0), BAD), (dict(C=P + 1), BAD),
    (dict(expert_offsets=0), BAD), (dict(status=0), BAD), (dict(workspace=0), BAD),
    (dict(workspace=P + 8), BAD), (dict(workspace_bytes=0), BAD), (dict(max_rows=0), BAD),
    (dict(max_rows=1 << 31), BAD), (dict(group_size=16), BAD), (dict(group_size=256), BAD),
    (dict(w_format=2), BAD), (dict(w_format=ep.EP_W4_E2M1), BAD),
    (dict(w_format=ep.EP_W4_E2M1, group_size=32, w_zeros=P), BAD),
    (dict(local_activation=2), BAD),
])
def test_w4_refusals(kw, code):
    assert call("ep_matvec_w4", cfg(), w4_args(**kw)) == code


def test_w4_shape_rules():
    assert call("ep_matvec_w4", cfg(K=80), w4_args()) == UNSUP
    assert call("ep_matvec_w4", cfg(K=96), w4_args()) == BAD  # groups of 64 in 96 columns
    assert call("ep_matvec_w4", cfg(N=129), w4_args(local_activation=ep.EP_ACT_SWIGLU)) == BAD
    assert call("ep_matvec_w4", cfg(dtype=ep.EP_FP8_1D2D), w4_args()) == UNSUP
    a = w4_args(A=0, gather_idx=P)
    a.x_ptrs[0] = P
    assert call("ep_matvec_w4", cfg(), a) == BAD  # the second rank's tokens are missing
    a.x_ptrs[1] = P + 8
    assert call("ep_matvec_w4", cfg(), a) == BAD
    assert call("ep_matvec_w4", cfg(n_ranks=9), w4_args()) == UNSUP
    n = ctypes.c_int64(0)
    assert ep.raw_call("ep_matvec_w4_sizes", ctypes.byref(cfg()), None) == BAD
    assert ep.raw_call("ep_matvec_w4_sizes", ctypes.byref(cfg(top_k=0)), ctypes.byref(n)) == BAD
    assert ep.ep_matvec_w4_sizes(cfg()) > 0


def test_binding_raises_with_the_code():
    with pytest.raises(ep.EpError) as e:
        ep.ep_route(cfg(), route_args(group_top=7))
    assert e.value.code == BAD and "ep_route" in str(e.value)


def test_argument_layouts_match_the_header(tmp_path):
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = [ep.ep_route_args, ep.ep_route_backward_args, ep.ep_combine_backward_args,
               ep.ep_w4_args]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe_ep.h"', "int main(void) {"]
    want = []
    for cls in structs:
        n = cls.__name__
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
        want.append(f"{n} {ctypes.sizeof(cls)}")
        for field, _ in cls._fields_:
            lines.append(f'printf("{n} {field} %zu %zu\\n", offsetof({n}, {field}), '
                         f'sizeof((({n} *)0)->{field}));')
            d = getattr(cls, field)
            want.append(f"{n} {field} {d.offset} {d.size}")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert [g for g in got if g] == want
