"""Arguments of the norm, its gradient, the 8-bit activation and the layer of a few tokens: layouts
against the header, refusals before any launch (no GPU)."""

import ctypes
import os
import shutil
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
                max_tokens_per_rank=100000, K=256, N=128, dtype=ep.EP_BF16, send_warps=-1,
                signal_mode=0)
    base.update(kw)
    return ep.ep_config(msg_bytes=2 * base["N"], **base)


def call(name, c, a):
    return ep.raw_call(name, ctypes.byref(c) if c is not None else None,
                       ctypes.byref(a) if a is not None else None, None)


def norm_args(**kw):
    base = dict(x=P, residual=P, residual_dtype=ep.EP_ROWS_F32, weight=P,
                weight_dtype=ep.EP_ROWS_BF16, eps=1e-6, hidden=128, sum=P, y=P, q=P, q_scales=P)
    base.update(kw)
    return ep.ep_add_rmsnorm_args(**base)


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(weight=0), dict(sum=0, y=0, q=0, q_scales=0), dict(q=0), dict(q_scales=0),
    dict(x=P + 1), dict(residual=P + 2), dict(sum=P + 2), dict(y=P + 1), dict(weight=P + 1),
    dict(q_scales=P + 2), dict(residual_dtype=2), dict(weight_dtype=-1), dict(hidden=0),
    dict(hidden=-8), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x_stride=127), dict(residual_stride=-1), dict(sum_stride=1), dict(y_stride=1 << 31),
])
def test_norm_refusals(kw):
    assert call("ep_add_rmsnorm", cfg(), norm_args(**kw)) == BAD


def test_norm_limits():
    assert call("ep_add_rmsnorm", cfg(), norm_args(hidden=ep.EP_MAX_NORM_HIDDEN + 1)) == UNSUP
    assert call("ep_add_rmsnorm", cfg(), None) == BAD
    assert call("ep_add_rmsnorm", None, norm_args()) == BAD
    assert call("ep_add_rmsnorm", cfg(num_tokens=0), norm_args(x=0, sum=0, y=0, q=0)) == ep.EP_OK


def back_args(**kw):
    base = dict(h=P, h_dtype=ep.EP_ROWS_F32, dy=P, dsum=P, weight=P, weight_dtype=ep.EP_ROWS_F32,
                eps=1e-6, hidden=128, dh=P, dx=P, dweight=P, workspace=P, workspace_bytes=1 << 40)
    base.update(kw)
    return ep.ep_add_rmsnorm_backward_args(**base)


@pytest.mark.parametrize("kw", [
    dict(h=0), dict(dy=0), dict(weight=0), dict(dh=0, dx=0, dweight=0), dict(h=P + 2),
    dict(dy=P + 1), dict(dsum=P + 2), dict(dh=P + 2), dict(dx=P + 1), dict(dweight=P + 2),
    dict(weight=P + 2), dict(h_dtype=3), dict(weight_dtype=2), dict(hidden=0), dict(eps=-1.0),
    dict(workspace=0), dict(workspace=P + 8), dict(workspace_bytes=64), dict(h_stride=100),
    dict(dy_stride=100), dict(dsum_stride=100), dict(dh_stride=100), dict(dx_stride=100),
])
def test_norm_backward_refusals(kw):
    assert call("ep_add_rmsnorm_backward", cfg(), back_args(**kw)) == BAD


def test_norm_backward_limits():
    c, n = cfg(), ctypes.c_int64(0)
    assert call("ep_add_rmsnorm_backward", c, back_args(hidden=16385)) == UNSUP
    assert call("ep_add_rmsnorm_backward", cfg(num_tokens=0), back_args(h=0, dweight=0)) == ep.EP_OK
    sizes = lambda c, hidden, out: ep.raw_call("ep_add_rmsnorm_backward_sizes", ctypes.byref(c),
                                               ctypes.c_int32(hidden), out)
    assert sizes(c, 0, ctypes.byref(n)) == BAD
    assert sizes(c, 128, None) == BAD
    assert sizes(c, 16385, ctypes.byref(n)) == UNSUP
    assert sizes(cfg(top_k=0), 128, ctypes.byref(n)) == BAD
    # enough for the largest call, and no less for fewer tokens than the call then has
    assert 0 < ep.ep_add_rmsnorm_backward_sizes(cfg(num_tokens=1), 128) \
        <= ep.ep_add_rmsnorm_backward_sizes(cfg(num_tokens=100000), 128)


def swiglu_args(**kw):
    base = dict(G=P, q=P, q_scales=P, expert_offsets=P, max_rows=64, inter=136)
    base.update(kw)
    return ep.ep_swiglu_e4m3_args(**base)


@pytest.mark.parametrize("kw", [
    dict(G=0), dict(q=0), dict(q_scales=0), dict(expert_offsets=0), dict(G=P + 8), dict(q=P + 4),
    dict(q_scales=P + 2), dict(expert_offsets=P + 2), dict(max_rows=0), dict(max_rows=1 << 31),
    dict(inter=0), dict(inter=4), dict(inter=132),
])
def test_swiglu_refusals(kw):
    assert call("ep_swiglu_e4m3", cfg(), swiglu_args(**kw)) == BAD


def test_swiglu_limit():
    assert call("ep_swiglu_e4m3", cfg(), swiglu_args(inter=(1 << 28) + 8)) == UNSUP
    assert call("ep_swiglu_e4m3", cfg(), swiglu_args(inter=1 << 30)) == UNSUP


def few_args(**kw):
    base = dict(x=P, x_scales=P, topk_ids=P, gates=P, W1=P, w1_scales=P, W2=P, w2_scales=P, out=P,
                workspace=P, workspace_bytes=1 << 40, status=P)
    base.update(kw)
    return ep.ep_layer_few_args(**base)


@pytest.mark.parametrize("dtype", [ep.EP_BF16, ep.EP_FP8_1D2D])
@pytest.mark.parametrize("kw", [
    dict(x=0), dict(topk_ids=0), dict(gates=0), dict(W1=0), dict(W2=0), dict(out=0),
    dict(workspace=0), dict(status=0), dict(x=P + 8), dict(W1=P + 8), dict(W2=P + 8),
    dict(workspace=P + 8), dict(out=P + 1), dict(topk_ids=P + 2), dict(gates=P + 2),
    dict(status=P + 2), dict(workspace_bytes=0),
])
def test_few_refusals(kw, dtype):
    assert call("ep_layer_few", cfg(dtype=dtype), few_args(**kw)) == BAD


@pytest.mark.parametrize("name", ["x_scales", "w1_scales", "w2_scales"])
def test_few_scales(name):
    for at in (0, P + 2):
        assert call("ep_layer_few", cfg(dtype=ep.EP_FP8_1D2D), few_args(**{name: at})) == BAD


@pytest.mark.parametrize("kw", [
    dict(num_tokens=65), dict(n_local_experts=64, top_k=33), dict(K=252), dict(N=132),
    dict(dtype=ep.EP_FP8_1D2D, K=320), dict(dtype=ep.EP_FP8_1D2D, N=192), dict(n_ranks=9),
    dict(K=1 << 30), dict(n_local_experts=256, K=1 << 26, N=1 << 24), dict(K=1 << 19, N=1 << 19),
    dict(dtype=ep.EP_FP8_1D2D, K=1 << 20, N=1 << 19),
])
def test_few_limits(kw):
    n = ctypes.c_int64(0)
    assert call("ep_layer_few", cfg(**kw), few_args()) == UNSUP
    assert ep.raw_call("ep_layer_few_sizes", ctypes.byref(cfg(**kw)), ctypes.byref(n)) == UNSUP


def test_few_sizes():
    assert ep.raw_call("ep_layer_few_sizes", ctypes.byref(cfg()), None) == BAD
    assert call("ep_layer_few", cfg(), None) == BAD
    assert call("ep_layer_few", cfg(num_tokens=0), few_args(x=0, out=0)) == ep.EP_OK
    assert ep.ep_layer_few_sizes(cfg()) > 0
    with pytest.raises(ep.EpError) as e:
        ep.ep_layer_few(cfg(), few_args(x=0))
    assert e.value.code == BAD and "ep_layer_few" in str(e.value)


def test_argument_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = [ep.ep_add_rmsnorm_args, ep.ep_add_rmsnorm_backward_args, ep.ep_swiglu_e4m3_args,
               ep.ep_layer_few_args]
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
