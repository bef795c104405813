"""Kernels that start while the one before them on the stream runs read nothing through the read-only path:
that is for what nobody writes as long as the kernel lives, and its loads need not stay behind the
kernel's wait for what the other one writes. Read off the sources: no run shows the order reliably."""

import os
import re

import pytest

from test_launch_order import CSRC

SOURCES = ["ep_combine.cu", "ep_combine_backward.cu", "ep_gemm_send.cu", "ep_gemm_send_fp8.cu",
           "ep_gemm_send_pair.cu", "ep_layer_few.cu", "ep_matvec_w4.cu", "ep_matvec_w4_wide.cu", "ep_norm.cu",
           "ep_route.cu", "ep_swiglu_e4m3.cu"]
HEADERS = ["ep_ptx.cuh", "ep_rows.cuh", "ep_sink.cuh", "ep_w4.cuh", "ep_w4_scales.cuh"]


def source_of(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_the_kernels_that_wait():
    waiting = [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "griddep_wait()" in source_of(f)]
    assert waiting == SOURCES
    included = {h for f in SOURCES + HEADERS for h in re.findall(r'#include "(\w+\.cuh)"', source_of(f))}
    assert included == set(HEADERS)


@pytest.mark.parametrize("source", SOURCES + HEADERS)
def test_no_read_only_loads_behind_the_wait(source):
    text = source_of(source)
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", text)
