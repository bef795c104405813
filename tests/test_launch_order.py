"""Kernels that are launched behind the one before them on the stream (programmatic dependent
launch) let their own dependents start only once everything before them has completed, so that
a dependent that does not wait, the combine whose inputs are ready, has no more than one
unfinished kernel before it. And no kernel ends before the one it was launched behind: what
waits for the combine waits for what the combine did not wait for. Read off the sources, as no
run can show the order reliably."""

import os
import re

import pytest

import moe_expert_gemm_gb300 as ep

CSRC = os.path.join(os.path.dirname(os.path.abspath(ep.__file__)), "csrc")


def kernels(path):
    """(name, body) of every __global__ function, comments left out."""
    src = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:const|C)", src):
        depth, i = 0, src.index("{", m.end())
        for j in range(i, len(src)):
            depth += (src[j] == "{") - (src[j] == "}")
            if depth == 0:
                yield m.group(1), src[i:j]
                break


SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


@pytest.mark.parametrize("source", SOURCES)
def test_dependents_start_after_the_wait(source):
    for name, body in kernels(os.path.join(CSRC, source)):
        if "griddep_launch_dependents()" not in body:
            continue
        assert "griddep_wait()" in body, name
        assert body.index("griddep_wait()") < body.index("griddep_launch_dependents()"), name


def test_the_kernels_are_found():
    found = [n for f in SOURCES for n, b in kernels(os.path.join(CSRC, f)) if "griddep_launch" in b]
    for name in ("route_token_kernel", "route_warp_kernel", "route_thread_kernel",
                 "route_backward_kernel", "route_backward_warp_kernel", "combine_backward_kernel",
                 "matvec_w4_kernel", "matvec_w4_wide_kernel"):
        assert name in found, (name, found)


def test_the_combine_ends_after_the_kernel_before_it():
    """In each of its kernels, ahead of every way out."""
    combines = list(kernels(os.path.join(CSRC, "ep_combine.cu")))
    assert len(combines) == 3
    for name, body in combines:
        ends = [m.start() for m in re.finditer(r"\breturn;", body)] + [len(body)]
        for end in ends:
            before = body[:end].rstrip()
            assert before.endswith("end_after_previous();"), (name, before[-80:])
