"""Routing calls of several host threads at once, each on a stream of its own, with numbers of experts that
take different amounts of the same kernel's shared memory."""

import threading

import pytest
import torch

import moe_expert_gemm_gb300 as ep

from test_gpu_route import cfg

pytestmark = pytest.mark.gpu


def test_calls_of_several_threads():
    T, k, calls = 64, 8, []
    for i, E in enumerate([2048, 1200, 2048, 1200]):
        x = torch.randn(T, E, generator=torch.Generator().manual_seed(i)).cuda()
        ids, gates = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
        a = ep.ep_route_args(logits=ep.ptr(x), logits_dtype=ep.EP_LOGITS_F32, score=ep.EP_SCORE_SOFTMAX,
                             n_groups=1, topk_groups=1, group_top=1, renormalize=1, scale=1.0,
                             topk_ids=ep.ptr(ids), gates=ep.ptr(gates))
        calls.append((cfg(T, E, k), a, torch.cuda.Stream(), x, ids, gates))
    torch.cuda.synchronize()
    alone = []
    for c in calls:
        ep.ep_route(*c[:3])
        torch.cuda.synchronize()
        order = c[3].sort(descending=True, stable=True).indices  # (equal logits go to the lower id)
        assert torch.equal(c[4], order[:, :k].int())
        alone.append((c[4].clone(), c[5].clone()))
    errors, start = [], threading.Barrier(len(calls))

    def run(c):
        start.wait()
        try:
            for _ in range(3000):
                ep.ep_route(*c[:3])
        except RuntimeError as e:
            errors.append(str(e))

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c, (ids, gates) in zip(calls, alone):
        assert torch.equal(c[4], ids) and torch.equal(c[5], gates)
