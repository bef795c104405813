"""No block ends while copies into its shared memory are in flight: whichever of its warps gave up, the
thread that issued them waits for the last copies into every stage. Read off the sources: no run shows
where the bytes of a copy land after its block has ended."""

import os
import re

import pytest

from test_launch_order import CSRC, kernels


def enclosing(body, at):
    """Heads of the blocks around position `at`, the outermost first."""
    heads, start = [], 0
    for i, c in enumerate(body[:at]):
        if c in ";{}":
            if c == "{":
                heads.append(" ".join(body[start:i].split()))
            elif c == "}":
                heads.pop()
            start = i + 1
    return heads


def statement(body, at):
    """From the end of the statement before position `at`, so that an unbraced `if` counts."""
    start = max(body.rfind(c, 0, at) for c in ";{}")
    return " ".join(body[start + 1:at].split())


# (kernel, source)
RINGS = [("few_kernel", "ep_layer_few.cu"), ("matvec_w4_kernel", "ep_matvec_w4.cu"),
         ("matvec_w4_wide_kernel", "ep_matvec_w4_wide.cu")]


@pytest.mark.parametrize("name,source", RINGS)
def test_the_producer_waits_whether_or_not_it_gave_up(name, source):
    body = dict(kernels(os.path.join(CSRC, source)))[name]
    calls = [m.start() for m in re.finditer(r"wait_for_copies<kStages>\(sh\.full, issued,", body)]
    assert len(calls) == 1
    heads = enclosing(body, calls[0])
    assert heads[0] == "" and len(heads) > 1  # the function, the producer's branch
    for head in heads + [statement(body, calls[0])]:
        assert not re.search(r"\bok\b", head), head
    # on every way out
    issued = body[:calls[0]].rfind("int issued = 0;")
    assert issued > 0 and not re.search(r"\breturn;", body[issued:calls[0]])


@pytest.mark.parametrize("name,source", [("few_kernel", "ep_layer_few.cu"), ("gemm_send_bf16_kernel", "ep_gemm_send.cu"),
                                         ("gemm_send_fp8_kernel", "ep_gemm_send_fp8.cu"),
                                         ("gemm_send_bf16_pair_kernel", "ep_gemm_send_pair.cu")])
def test_a_calls_short_limit_does_not_cut_that_wait(name, source):
    """The limit of a call's waits may be a nanosecond; what a block has under way ends all the same: waits that
    nobody may abort have a limit of their own."""
    body = dict(kernels(os.path.join(CSRC, source)))[name]
    waits = re.findall(r"\w+_wait\w*\(([^;]*?)&no_abort\)", body) + re.findall(r"wait_for_copies<\w+>\(([^;]*?)\);", body)
    assert len(waits) == 2, waits
    for args in waits:
        assert "kEndNs" in args and "p.timeout_ns" not in args, args
