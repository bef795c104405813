"""The second kernel of the layer of a few tokens starts while the first one runs. No wait with a limit
begins before the first one has ended, however long it takes: read off the source."""

import os
import re

from test_launch_order import CSRC, kernels


def test_limits_count_from_the_first_kernels_end():
    body = dict(kernels(os.path.join(CSRC, "ep_layer_few.cu")))["few_kernel"]
    starts = [m.start() for m in re.finditer(r"\bif \(warp == 0\)|else if \([^)]*warp", body)]
    branches = [body[a:b] for a, b in zip(starts, starts[1:] + [len(body)])]
    waiting = [b for b in branches if re.search(r"\bmbar_wait\(", b)]
    assert len(waiting) == 4  # copies, products, sums, scales
    for b in waiting:
        assert "griddep_wait()" in b and b.index("griddep_wait()") < re.search(r"\bmbar_wait\(", b).start()
