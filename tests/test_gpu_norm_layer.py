"""The norm, the router, the layer of a few tokens, the fp8 layer and the gradients as EpSystem runs
them one after the other: against the formulas in 64 bits and against each other."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
import rows_reference as ref
from moe_expert_gemm_gb300.system import EpSystem
from moe_expert_gemm_gb300.w4 import quantize_w4
from rows_reference import BF16, F32

pytestmark = pytest.mark.gpu

R, EL, K_TOP, H, I = 2, 4, 3, 512, 256
E = R * EL


def codes_of(w):
    """e4m3 codes and block scales of [E][N][K]."""
    e, n, k = w.shape
    b = w.view(e, n // 128, 128, k // 128, 128)
    s = b.abs().amax((2, 4)) / 448
    return (b / s[:, :, None, :, None]).view(e, n, k).to(torch.float8_e4m3fn).cuda(), s.cuda()


class Block:
    """A rank group's tokens, weights and buffers; `run` is a block of a model: norm, router, layer."""

    def __init__(self, tokens, fp8, seed):
        gen = torch.Generator().manual_seed(seed)
        self.rand = lambda *shape: torch.randn(*shape, generator=gen)
        self.T, self.fp8 = tokens, fp8
        self.s = EpSystem(R, EL, K_TOP, tokens, K=I, N=H, dtype="fp8_1d2d" if fp8 else "bf16")
        self.weight = (1 + 0.2 * self.rand(H)).cuda()
        self.router = (self.rand(E, H) / H ** 0.5).cuda()
        self.x, self.res, self.y, self.q, self.qs, self.parts, self.W = [], [], [], [], [], [], []
        for r in range(R):
            self.x.append(self.rand(tokens, H).cuda().bfloat16())
            self.res.append(self.rand(tokens, H).cuda())
            self.y.append(torch.zeros(tokens, H, dtype=torch.bfloat16, device="cuda"))
            self.q.append(torch.zeros(tokens, H, dtype=torch.float8_e4m3fn, device="cuda"))
            self.qs.append(torch.zeros(tokens, H // 128, device="cuda"))
            W1, W2 = self.rand(EL, 2 * I, H) / H ** 0.5, self.rand(EL, H, I) / I ** 0.5
            if fp8:
                self.W.append(codes_of(W1) + codes_of(W2))
            else:
                self.W.append((W1.bfloat16().cuda(), None, W2.bfloat16().cuda(), None))
            self.s.set_layer_few(r, self.W[r][0], self.W[r][2], self.W[r][1], self.W[r][3])
            self.parts.append([torch.zeros(tokens, H, dtype=torch.bfloat16, device="cuda") for _ in range(R)])

    def norm_and_route(self, stream=None):
        for r in range(R):
            self.s.add_rmsnorm(r, self.x[r], self.weight, residual=self.res[r], sum=self.res[r], y=self.y[r],
                               q=self.q[r], q_scales=self.qs[r], stream=stream)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            logits = [y.float() @ self.router.T for y in self.y]
        for r in range(R):
            self.s.route(r, logits[r], stream=stream)
        self.logits = logits

    def few(self, stream=None):
        """Every rank's part of every rank's tokens."""
        for r in range(R):
            for src in range(R):
                self.s.layer_few(r, self.q[src] if self.fp8 else self.y[src], self.parts[src][r],
                                 x_scales=self.qs[src] if self.fp8 else None, source=src, stream=stream)

    def long_way(self, epoch=1, stream=None):
        """Plan, dispatch, grouped products, combine."""
        for r in range(R):
            self.s.plan(r, stream=stream)
        for r in range(R):
            if self.fp8:
                self.s.set_layer_fp8(r, self.q[r], self.qs[r], *self.W[r])
            else:
                bits = lambda t: t.cpu().view(torch.int16).numpy()
                self.s.set_layer_operands(r, bits(self.y[r]), bits(self.W[r][0]), bits(self.W[r][2]))
        for r in range(R):
            if self.fp8:
                self.s.layer_forward_fp8(r, epoch, stream)
            else:
                self.s.layer_forward(r, epoch, stream, fused_act=True)
        for r in range(R):
            self.s.combine(r, epoch, stream=stream)

    def values(self, r):
        if self.fp8:
            return ref.wide_blocks(self.W[r][0], self.W[r][1]), ref.wide_blocks(self.W[r][2], self.W[r][3])
        return self.W[r][0].double(), self.W[r][2].double()

    def reference(self, src, r):
        W1, W2 = self.values(r)
        x = ref.wide(self.q[src], self.qs[src]) if self.fp8 else self.y[src].double()
        return ref.layer_few(x, self.s.topk[src], self.s.gates[src], W1, W2, r * EL, self.fp8)


@pytest.mark.parametrize("tokens", [1, 19, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_block_of_a_model(tokens, fp8):
    b = Block(tokens, fp8, seed=tokens)
    x, res = [v.clone() for v in b.x], [v.clone() for v in b.res]
    b.norm_and_route()
    b.few()
    torch.cuda.synchronize()
    assert (b.s.status_words() == 0).all()
    for r in range(R):
        h, v = ref.norm(x[r], res[r], b.weight, 1e-6)
        assert ((b.res[r].double() - h).abs() <= 2 * F32 * h.abs()).all()
        assert ((b.y[r].double() - v).abs() <= (BF16 + 48 * F32) * v.abs()).all()
        ref.check_e4m3(b.q[r], b.qs[r], v, 48 * F32)
    for src in range(R):
        for r in range(R):
            want, bound = b.reference(src, r)
            got = b.parts[src][r].double().cpu()
            assert ((got - want).abs() <= BF16 * (want.abs() + bound) + bound).all()
    # the long way: rows rounded to bf16 (and, fp8, the up/gate rows), then the sum. The two agree to
    # within those roundings of the magnitudes that are summed
    b.long_way()
    torch.cuda.synchronize()
    assert (b.s.status_words() == 0).all()
    for src in range(R):
        parts = torch.stack([p.double() for p in b.parts[src]])
        total, size = parts.sum(0), torch.zeros(tokens, H, dtype=torch.float64, device="cuda")
        x_of = ref.wide(b.q[src], b.qs[src]) if fp8 else b.y[src].double()
        for t in range(tokens):
            for j in range(K_TOP):
                e = int(b.s.topk[src][t, j])
                W1, W2 = b.values(e // EL)
                a = ref.swiglu(W1[e % EL] @ x_of[t])
                size[t] += b.s.gates[src][t, j].double() * (W2[e % EL] @ a).abs()
        off = (b.s.out[src].double() - total).norm()
        # Long way: rows and their sum rounded, few: each part, three times BF16 of the size in all. bf16: both
        # round the same fp32 activation, a few to different neighbours (a quarter more). fp8: the long way
        # rounds the up/gate rows to bf16, which moves an activation by up to d = 2.1 BF16 of itself; a code
        # then moves by a step (2^-3 at most) with the chance d / step, sqrt(2^-3 d) = 8.2 BF16 in the
        # root of the mean square, in which the products pass it on.
        assert off <= (12 if fp8 else 4) * BF16 * size.norm()


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_replayed(fp8):
    """The block captured once: replays on other tokens give the bits of single calls."""
    b, one = Block(10, fp8, seed=3), Block(10, fp8, seed=3)
    stream = torch.cuda.Stream()

    def step(k, st):
        k.norm_and_route(st)
        k.few(st)

    step(b, stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(b, torch.cuda.current_stream())
    for seed in (1, 2, 3):
        gen = torch.Generator().manual_seed(seed)
        for r in range(R):
            x, res = torch.randn(10, H, generator=gen), torch.randn(10, H, generator=gen)
            for k in (b, one):
                k.x[r].copy_(x)
                k.res[r].copy_(res)
        torch.cuda.synchronize()
        graph.replay()
        step(one, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert (b.s.status_words() == 0).all() and (one.s.status_words() == 0).all()
        for src in range(R):
            assert torch.equal(b.res[src], one.res[src]) and torch.equal(b.y[src], one.y[src])
            assert torch.equal(b.s.topk[src], one.s.topk[src])
            for r in range(R):
                assert torch.equal(b.parts[src][r], one.parts[src][r])


def test_behind_a_busy_current_stream():
    """Calls on a stream of their own while torch's current one is busy: nothing that a call makes
    for itself may be left to that one."""
    b = Block(12, False, seed=4)
    stream = torch.cuda.Stream()
    dy = torch.randn(12, H, generator=torch.Generator().manual_seed(0)).cuda().bfloat16()
    dh, dw = torch.zeros(12, H, device="cuda"), torch.zeros(H, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    b.norm_and_route(stream)
    b.few(stream)
    b.s.add_rmsnorm_backward(0, b.res[0], dy, b.weight, dh=dh, dweight=dw, stream=stream.cuda_stream)
    stream.synchronize()
    got = [b.parts[0][0].clone(), dh.clone(), dw.clone()]
    torch.cuda.synchronize()
    want, bound = b.reference(0, 0)
    assert ((got[0].double().cpu() - want).abs() <= BF16 * (want.abs() + bound) + bound).all()
    want, want_w, size, size_w = ref.norm_backward(b.res[0], dy, b.weight, None, 1e-6)
    assert ((got[1].double() - want).abs() <= 256 * F32 * size + F32 * want.abs()).all()
    assert ((got[2].double() - want_w).abs() <= 128 * F32 * size_w).all()


def test_training_through_the_norm():
    """The gradient of a router behind the norm, down to the norm's input and weight: the layer on 4-bit
    weights, the combine's and the router's gradients, then the norm's."""
    T = 24
    gen = torch.Generator().manual_seed(9)
    s = EpSystem(R, EL, K_TOP, T, K=I, N=H)
    weight, router = (1 + 0.1 * torch.randn(H, generator=gen)).cuda(), (torch.randn(E, H, generator=gen) / H ** 0.5).cuda()
    x = [torch.randn(T, H, generator=gen).cuda().bfloat16() for _ in range(R)]
    res = [torch.randn(T, H, generator=gen).cuda() for _ in range(R)]
    y = [torch.zeros_like(v) for v in x]
    logits = []
    for r in range(R):
        s.add_rmsnorm(r, x[r], weight, residual=res[r], sum=res[r], y=y[r])
        s.set_layer_w4(r, y[r], quantize_w4(torch.randn(EL, 2 * I, H, generator=gen).cuda() / H ** 0.5),
                       quantize_w4(torch.randn(EL, H, I, generator=gen).cuda() / I ** 0.5))
        logits.append(y[r].float() @ router.T)
        s.route(r, logits[r])
    for r in range(R):
        s.plan(r)
        s.layer_forward_w4(r, epoch=1)
    for r in range(R):
        s.combine(r, epoch=1)
    total_w = torch.zeros(H, dtype=torch.float64, device="cuda")
    for r in range(R):
        dout = torch.randn(T, H, generator=gen).cuda().bfloat16()
        dgates, dlogits = torch.zeros(T, K_TOP, device="cuda"), torch.zeros(T, E, device="cuda")
        dh, dw, dx = torch.zeros(T, H, device="cuda"), torch.zeros(H, device="cuda"), torch.zeros_like(x[r])
        s.combine_backward(r, dout, dgates=dgates)
        s.route_backward(r, dgates, dlogits)
        dy = (dlogits @ router).bfloat16()
        s.add_rmsnorm_backward(r, res[r], dy, weight, dsum=dout.float(), dh=dh, dx=dx, dweight=dw)
        torch.cuda.synchronize()
        assert (s.status_words() == 0).all()
        # automatic differentiation of the norm in 64 bits
        h, w = res[r].double().requires_grad_(True), weight.double().requires_grad_(True)
        v = h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w
        (v * dy.double()).sum().backward()
        _, _, size, size_w = ref.norm_backward(res[r], dy, weight, dout.float(), 1e-6)
        assert ((dh.double() - h.grad - dout.double()).abs() <= 256 * F32 * size).all()
        assert ((dx.double() - h.grad - dout.double()).abs() <= BF16 * (h.grad + dout.double()).abs() + 260 * F32 * size).all()
        assert ((dw.double() - w.grad).abs() <= 128 * F32 * size_w).all()
        total_w += dw.double()
    assert total_w.norm() > 0


def test_no_tokens():
    s = EpSystem(1, EL, 2, 0, K=I, N=H, max_tokens=4)
    empty = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype, device="cuda")
    w, dw = torch.ones(H, device="cuda"), torch.ones(H, device="cuda")
    s.add_rmsnorm(0, empty(0, H), w, residual=empty(0, H), sum=empty(0, H), y=empty(0, H))
    s.add_rmsnorm_backward(0, empty(0, H), empty(0, H), w, dh=empty(0, H), dweight=dw)
    s.route(0, empty(0, EL, dtype=torch.float32))
    s.set_layer_few(0, empty(EL, 2 * I, H), empty(EL, H, I))
    s.layer_few(0, empty(0, H), empty(0, H))
    torch.cuda.synchronize()
    assert (s.status_words() == 0).all() and (dw == 0).all()
