"""The layer of a few tokens against its formula in 64 bits."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
import rows_reference as ref
from rows_reference import BF16

pytestmark = pytest.mark.gpu


class Few:
    """Operands of one call, and the call."""

    def __init__(self, T, E, k, H, I, fp8=False, R=1, rank=0, seed=0, ids=None):
        gen = torch.Generator().manual_seed(seed)
        self.fp8, self.first, self.T, self.H = fp8, rank * E, T, H
        self.cfg = ep.ep_config(R, rank, E, k, T, max(T, 1), I, H, 2 * H, ep.EP_FP8_1D2D if fp8 else ep.EP_BF16,
                                -1, 0)
        x = torch.randn(T, H, generator=gen)
        W1 = torch.randn(E, 2 * I, H, generator=gen) * H ** -0.5
        W2 = torch.randn(E, H, I, generator=gen) * I ** -0.5
        self.xs = self.w1s = self.w2s = None
        if fp8:
            self.x, self.xs = self.rows(x)
            self.W1, self.w1s = self.blocks(W1)
            self.W2, self.w2s = self.blocks(W2)
        else:
            self.x, self.W1, self.W2 = (v.bfloat16().cuda() for v in (x, W1, W2))
        if ids is None:
            ids = torch.rand(T, R * E, generator=gen).argsort(1)[:, :k]
        self.ids = ids.to(torch.int32).cuda().contiguous()
        self.gates = torch.softmax(torch.randn(T, k, generator=gen), -1).cuda()
        self.out = torch.full((T, H), torch.nan, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.size = ep.ep_layer_few_sizes(self.cfg)
        self.work = torch.zeros(self.size + 64, dtype=torch.uint8, device="cuda")
        self.work[self.size:] = 0x5A

    @staticmethod
    def rows(x):
        s = ref.scales(x).float()
        return (ref.groups(x) / s[..., None]).flatten(-2).to(torch.float8_e4m3fn).cuda(), s.cuda()

    @staticmethod
    def blocks(w):
        E, N, K = w.shape
        b = w.view(E, N // 128, 128, K // 128, 128)
        s = b.abs().amax((2, 4)) / 448
        return (b / s[:, :, None, :, None]).view(E, N, K).to(torch.float8_e4m3fn).cuda(), s.cuda()

    def call(self, stream=None, out=None, work=None):
        a = ep.ep_layer_few_args(x=ep.ptr(self.x), x_scales=ep.ptr(self.xs), topk_ids=ep.ptr(self.ids),
                                 gates=ep.ptr(self.gates), W1=ep.ptr(self.W1), w1_scales=ep.ptr(self.w1s),
                                 W2=ep.ptr(self.W2), w2_scales=ep.ptr(self.w2s),
                                 out=ep.ptr(self.out if out is None else out),
                                 workspace=ep.ptr(self.work if work is None else work),
                                 workspace_bytes=self.size, status=ep.ptr(self.status))
        ep.ep_layer_few(self.cfg, a, stream)

    def reference(self):
        if self.fp8:
            v = ref.wide(self.x, self.xs), ref.wide_blocks(self.W1, self.w1s), ref.wide_blocks(self.W2, self.w2s)
        else:
            v = self.x.double(), self.W1.double(), self.W2.double()
        return ref.layer_few(v[0], self.ids, self.gates, v[1], v[2], self.first, self.fp8)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status) == status
        assert (self.work[self.size:] == 0x5A).all()
        want, bound = self.reference()
        got = self.out.double().cpu()
        assert ((got - want).abs() <= BF16 * (want.abs() + bound) + bound).all()
        # as a whole: out's rounding is at most BF16 of it; activations that the two round to
        # different neighbours are few (where an fp32 sum's error crosses a tie), BF16 / 4 for them
        if want.norm() > 0:
            assert (got - want).norm() <= 1.25 * BF16 * want.norm()


SIZES = [
    # T, E, k, H, I
    (1, 8, 2, 128, 256), (1, 1, 1, 8, 8), (1, 4, 4, 64, 72), (2, 3, 2, 136, 264), (5, 12, 3, 248, 200),
    (7, 1, 1, 1000, 504), (16, 16, 4, 256, 128), (17, 5, 5, 512, 640), (33, 9, 2, 328, 96), (64, 6, 3, 384, 256),
    (64, 64, 8, 128, 128), (48, 256, 6, 64, 64), (3, 2, 1, 2056, 1000), (1, 4, 2, 1000, 4104), (64, 2, 2, 264, 1016),
    (64, 256, 32, 64, 64), (63, 8, 8, 72, 136),
]
SIZES_8 = [(1, 8, 2, 128, 256), (1, 1, 1, 128, 128), (5, 12, 3, 256, 384), (16, 16, 4, 384, 128),
           (17, 5, 5, 512, 640), (33, 9, 2, 128, 1152), (64, 6, 3, 384, 256), (64, 64, 8, 128, 128),
           (2, 3, 2, 2176, 256), (1, 4, 2, 256, 4224), (64, 2, 2, 640, 896), (64, 256, 32, 128, 128)]


@pytest.mark.parametrize("T,E,k,H,I", SIZES)
def test_bf16(T, E, k, H, I):
    f = Few(T, E, k, H, I, seed=T + H)
    f.call()
    f.check()


@pytest.mark.parametrize("T,E,k,H,I", SIZES_8)
def test_e4m3(T, E, k, H, I):
    f = Few(T, E, k, H, I, fp8=True, seed=T + H)
    f.call()
    f.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_the_ranks_parts(fp8):
    """Each rank's part against the formula; a token without an expert here gets zeros."""
    for rank in range(3):
        f = Few(9, 4, 2, 256, 384, fp8=fp8, R=3, rank=rank, seed=5)
        f.call()
        f.check()
        here = ((f.ids >= 4 * rank) & (f.ids < 4 * rank + 4)).any(1)
        assert (f.out[~here] == 0).all() and (~here).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_no_token_has_an_expert_here(fp8):
    f = Few(6, 3, 2, 256, 128, fp8=fp8, R=2, rank=1, ids=torch.tensor([[0, 2]] * 6))
    f.call()
    f.check()
    assert (f.out == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_same_expert_twice_and_ids_outside(fp8):
    ids = torch.tensor([[0, 0, 1], [2, 1, 2], [-1, 3, 0], [7, 4, 100], [-2 ** 31, 2 ** 31 - 1, 5], [3, 3, 3]])
    f = Few(6, 5, 3, 256, 128, fp8=fp8, ids=ids, seed=2)
    f.call()
    f.check(status=ep.EP_STATUS_ROUTING)
    assert (f.out[4] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 20, 64])
def test_every_token_to_one_expert(fp8, T):
    f = Few(T, 200, 1, 128, 256, fp8=fp8, ids=torch.full((T, 1), 131), seed=3)
    f.call()
    f.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_infinities_and_nan_stay_with_their_tokens(fp8):
    """Of experts that a token does not use, of other tokens, of the workspace."""
    T, E = 12, 6
    ids = torch.tensor([[t % 4, (t + 1) % 4] for t in range(T)])
    f = Few(T, E, 2, 256, 128, fp8=fp8, ids=ids, seed=4)
    f.call()
    torch.cuda.synchronize()
    clean = f.out.clone()
    f.W1[4:], f.W2[4:] = torch.nan, torch.nan  # nobody's experts
    if fp8:
        f.w1s[5], f.w2s[5] = torch.inf, torch.nan
        f.W2[1, 3, 7] = torch.nan
        f.xs[2, 0] = torch.nan
    else:
        f.W2[1, 3, 7] = torch.inf
        f.x[2, 5] = torch.nan
    f.gates[7, 1] = torch.inf
    f.call()
    torch.cuda.synchronize()
    assert int(f.status) == 0
    uses_1 = (f.ids == 1).any(1)
    same = torch.ones(T, 256, dtype=torch.bool, device="cuda")
    same[uses_1, 3] = False
    same[2] = same[7] = False
    assert torch.equal(f.out[same], clean[same])
    assert f.out[2].isnan().all()
    assert (~f.out[uses_1, 3].isfinite()).all()
    assert (~f.out[7].isfinite()).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_repeated_calls_and_streams(fp8):
    """The workspace is ready for the next call, also on another stream, and the bits are the same."""
    f = Few(20, 8, 3, 512, 384, fp8=fp8, seed=6)
    f.call()
    f.check()
    first = f.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(5):
        f.out.fill_(torch.nan)
        side.wait_stream(torch.cuda.current_stream())
        f.call(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(f.out, first)
    # two at once, with a workspace each
    other, work = torch.zeros_like(f.out), torch.zeros_like(f.work)
    torch.cuda.synchronize()
    for i in range(20):
        f.call()
        f.call(side, other, work)
    torch.cuda.synchronize()
    assert torch.equal(f.out, first) and torch.equal(other, first)
    assert int(f.status) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_and_replayed(fp8):
    f = Few(10, 8, 3, 512, 384, fp8=fp8, seed=7)
    f.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f.call(torch.cuda.current_stream())
        f.call(torch.cuda.current_stream())
    g = Few(10, 8, 3, 512, 384, fp8=fp8, seed=8)
    for name in ("x", "xs", "ids", "gates"):
        if getattr(f, name) is not None:
            getattr(f, name).copy_(getattr(g, name))
    f.out.fill_(torch.nan)
    for _ in range(3):
        graph.replay()
    f.check()


def test_out_at_any_element():
    f = Few(3, 4, 2, 136, 72, seed=9)
    out = torch.full((3 * 136 + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    f.out = out[1:1 + 3 * 136].view(3, 136)
    f.call()
    f.check()
    assert out[0] == 7 and (out[1 + 3 * 136:] == 7).all()


def test_no_tokens():
    f = Few(0, 4, 2, 128, 128)
    f.call()
    torch.cuda.synchronize()
    assert int(f.status) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_real_sizes(fp8):
    """A decode batch of real widths: sampled columns against the formula."""
    T, E, k, H, I = 16, 12, 4, 4096, 2048
    f = Few(T, E, k, H, I, fp8=fp8, seed=10)
    f.call()
    f.check()


def test_one_workspace_for_many_configurations():
    """Sized for the largest; what another configuration left in it does no harm."""
    work, outs = None, []
    for T, fp8 in [(64, False), (1, False), (20, True), (64, True), (33, False), (1, True), (5, False)]:
        f = Few(T, 9, 3, 384, 640, fp8=fp8, seed=T)
        if work is None:
            work = torch.zeros(f.size + 64, dtype=torch.uint8, device="cuda")
            work[f.size:] = 0x5A
            largest = f.size
        assert f.size <= largest
        f.call(work=work)
        f.check()
        assert (work[largest:] == 0x5A).all()
        work[4096:largest] = 0xFF  # NaN, in all but the counters


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_unwritten_is_used(fp8):
    """Results are the same with NaN in the workspace's sums and rows."""
    for T, E, k, H, I in [(11, 7, 2, 640, 384), (40, 3, 2, 128, 1152)]:
        f = Few(T, E, k, H, I, fp8=fp8, seed=12)
        f.work[4096:f.size] = 0xFF
        f.call()
        f.check()
