"""Kernels that start while the one before them on the stream runs read nothing through the read-only path:
that is for what nobody writes as long as the kernel lives, and its loads need not stay behind the
kernel's wait for what the other one writes. Read off the sources: no run shows the order reliably."""

import os
import re

import pytest

from test_launch_order import CSRC

SOURCES = ["ep_swiglu_e4m3.cu"]


@pytest.mark.parametrize("source", SOURCES)
def test_no_read_only_loads_behind_the_wait(source):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, source)).read())
    assert "griddep_wait()" in text
    assert not re.findall(r"__ldg\b|ld\.global\.nc|__restrict__", text)
