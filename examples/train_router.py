"""Trains the router of a MoE layer whose experts are frozen in 4 bits.

A step, every call on the device and none of them waiting: the router's logits, the choice
of the experts and their gates (ep_route), the plan, the experts' products on 4-bit weights
(ep_matvec_w4, twice), the scatter and the combine; then back from the squared distance
to given outputs to the gates (ep_combine_backward), to the logits (ep_route_backward) and to
the router's weights. The layer before and after, the router's own products and the
optimiser are PyTorch's.

    python examples/train_router.py --steps 60
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_gemm_gb300 as ep
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4


def train(steps=60, ranks=2, local_experts=8, top_k=4, tokens=64, hidden=512, inter=256,
          w_format=ep.EP_W4_E2M1, lr=0.3, momentum=0.9, seed=0, log=print):
    """Returns the loss of every step, summed over the ranks."""
    gen = torch.Generator("cpu").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen)
    E = ranks * local_experts
    s = EpSystem(ranks, local_experts, top_k, tokens, K=inter, N=hidden)
    X, target = [], []
    teacher = rand(E, hidden).cuda() * 2 / hidden ** 0.5
    for r in range(ranks):
        X.append(rand(tokens, hidden).cuda().bfloat16())
        w1 = rand(local_experts, 2 * inter, hidden).cuda() / hidden ** 0.5
        w2 = rand(local_experts, hidden, inter).cuda() * 2 / inter ** 0.5
        s.set_layer_w4(r, X[r], quantize_w4(w1, w_format), quantize_w4(w2, w_format))

    epoch = 0

    def forward(router):
        nonlocal epoch
        epoch += 1
        for r in range(ranks):
            s.route(r, X[r].float() @ router.T)
        for r in range(ranks):
            s.plan(r)
            s.layer_forward_w4(r, epoch)
        for r in range(ranks):
            s.combine(r, epoch)

    forward(teacher)  # what the layer answers with another router is what it is to learn
    target = [o.float() for o in s.out]
    router = teacher + rand(E, hidden).cuda() / hidden ** 0.5
    speed = torch.zeros_like(router)
    dgates = torch.empty(tokens, top_k, device="cuda")
    dlogits = torch.empty(tokens, E, device="cuda")
    losses = []
    for step in range(steps):
        forward(router)
        grad = torch.zeros_like(router)
        loss = 0
        for r in range(ranks):
            off = s.out[r].float() - target[r]
            loss = loss + off.square().mean()
            s.combine_backward(r, (off * (2 / tokens)).bfloat16(), dgates=dgates)
            s.route_backward(r, dgates, dlogits)
            grad += dlogits.T @ X[r].float()
        speed = momentum * speed + grad / hidden
        router = router - lr * speed
        losses.append(loss)
        if log and step % 10 == 0:
            log(f"step {step}: loss {float(loss):.5f}")
    losses = [float(v) for v in losses]
    if any(s.status_words()):
        raise RuntimeError(f"status words {s.status_words()}")
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--format", choices=("int", "e2m1"), default="e2m1")
    o = a.parse_args()
    losses = train(o.steps, w_format=ep.EP_W4_E2M1 if o.format == "e2m1" else ep.EP_W4_INT)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f}")
