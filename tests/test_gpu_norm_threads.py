"""Calls of the norm and its gradient from several host threads at once, each on a stream of its own: calls
of other sizes of the same kernel do not take a call's shared memory away between its set-up and its launch."""

import threading

import pytest
import torch

import moe_expert_gemm_gb300 as ep

from test_gpu_norm import ROWS, cfg

pytestmark = pytest.mark.gpu

# rows of four pieces a thread, whole pieces and not; (tokens, hidden)
FORMS = {"norm": [(400, 16384), (400, 8448)], "norm any": [(400, 16383), (400, 8449)],
         "gradient": [(400, 16384), (400, 8448)], "gradient any": [(400, 16383), (400, 8449)]}


class Call:
    """One call's operands, kept; `again` makes it."""

    def __init__(self, form, T, n, seed):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=gen).cuda().bfloat16()
        self.x, self.other, self.w, self.out = rand(T, n), rand(T, n), rand(n), torch.zeros(T, n).cuda().bfloat16()
        self.stream, self.cfg = torch.cuda.Stream(), cfg(T)
        common = dict(weight=ep.ptr(self.w), weight_dtype=ROWS[self.w.dtype], eps=1e-6, hidden=n)
        if form.startswith("norm"):
            self.f = ep.ep_add_rmsnorm
            self.a = ep.ep_add_rmsnorm_args(x=ep.ptr(self.x), residual=ep.ptr(self.other), y=ep.ptr(self.out),
                                            residual_dtype=ep.EP_ROWS_BF16, **common)
        else:
            self.f = ep.ep_add_rmsnorm_backward
            self.a = ep.ep_add_rmsnorm_backward_args(h=ep.ptr(self.x), dy=ep.ptr(self.other), dh=ep.ptr(self.out),
                                                     h_dtype=ep.EP_ROWS_BF16, **common)

    def again(self):
        self.f(self.cfg, self.a, self.stream)


@pytest.mark.parametrize("form", FORMS)
def test_calls_of_several_threads(form):
    calls = [Call(form, T, n, i) for i, (T, n) in enumerate(FORMS[form] * 2)]
    torch.cuda.synchronize()
    alone = []
    for c in calls:
        c.again()
        torch.cuda.synchronize()
        alone.append(c.out.clone())
    errors = []
    start = threading.Barrier(len(calls))

    def run(c):
        start.wait()
        try:
            for _ in range(2000):
                c.again()
        except RuntimeError as e:
            errors.append(str(e))

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c, want in zip(calls, alone):
        assert torch.equal(c.out, want)
