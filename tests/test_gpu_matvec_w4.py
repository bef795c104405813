"""Expert products on 4-bit weights on the GPU against the 64-bit reference.

Element by element: half the spacing of bf16 numbers (7 stored bits: 2^-8, plus what the SiLU's fp32
steps add, under 2^-20) and fp32 sums whose chains are at most K/16 + 64 long, at 2^-23
each (matrix instructions may cut instead of round) of sum |w||x|. Over all: correct
rounding keeps the relative 2-norm of the error under 2^-8; fp32 sums of random signs
stay far below the 2^-13 allowed beside it."""

import numpy as np
import pytest
import torch

import moe_expert_gemm_gb300 as ep
import operator_reference as ref

pytestmark = pytest.mark.gpu


def cfg(E, N, K, ranks=1, k=1, T=1):
    return ep.ep_config(n_ranks=ranks, my_rank=0, n_local_experts=E, top_k=k, num_tokens=T,
                        max_tokens_per_rank=max(T, 1), K=K, N=N, msg_bytes=2 * N,
                        dtype=ep.EP_BF16, send_warps=-1, signal_mode=0)


def weights(E, N, K, fmt, group, seed):
    rng = np.random.default_rng(seed)
    packed = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    shape = (E, N, K // group)
    if fmt == "e2m1":
        return packed, rng.integers(110, 135, shape).astype(np.uint8), None
    scales = ref.bf16_round((rng.random(shape) * 0.1 + 0.01).astype(np.float32))
    return packed, scales, rng.integers(0, 16, shape).astype(np.uint8) if fmt == "int4z" else None


class Call:
    """Device copies of one call's inputs; C and the workspace have guards behind them."""

    def __init__(self, x, counts, w, fmt, group, act=False, max_rows=None, offsets=None):
        self.packed, self.scales, self.zeros = w
        self.E, self.N, k2 = self.packed.shape
        self.K, self.fmt, self.group, self.act = 2 * k2, fmt, group, act
        self.x = x
        self.offsets = np.concatenate(([0], np.cumsum(counts))) if offsets is None else offsets
        self.max_rows = max_rows or max(1, int(sum(counts)))
        self.cols = self.N // 2 if act else self.N
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.W = dev(self.packed)
        self.S = dev(self.scales) if fmt == "e2m1" else dev(self.scales).to(torch.bfloat16)
        self.Z = None if self.zeros is None else dev(self.zeros)
        self.off = dev(self.offsets.astype(np.int32))
        rows = np.zeros((self.max_rows, self.K), np.float32)
        rows[:len(x)] = x
        rows[len(x):] = np.nan  # rows past the plan's count
        self.A = dev(rows).to(torch.bfloat16)
        self.C = torch.full((self.max_rows * self.cols + 64,), 55.0, dtype=torch.bfloat16, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cfg = cfg(self.E, self.N, self.K)
        n = ep.ep_matvec_w4_sizes(self.cfg)
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.args = ep.ep_w4_args(
            A=ep.ptr(self.A), W=ep.ptr(self.W), w_scales=ep.ptr(self.S), w_zeros=ep.ptr(self.Z),
            w_format=ep.EP_W4_E2M1 if fmt == "e2m1" else ep.EP_W4_INT, group_size=group,
            expert_offsets=ep.ptr(self.off), max_rows=self.max_rows,
            local_activation=ep.EP_ACT_SWIGLU if act else ep.EP_ACT_NONE, C=ep.ptr(self.C),
            workspace=ep.ptr(self.ws), workspace_bytes=n, status=ep.ptr(self.status))

    def run(self, stream=None):
        torch.cuda.synchronize()
        ep.ep_matvec_w4(self.cfg, self.args, stream)
        torch.cuda.synchronize()
        self.bits = self.C.view(torch.int16).cpu().numpy().copy()
        out = self.C.float().cpu().numpy().astype(np.float64)
        m = int(self.offsets[-1])
        assert (out[m * self.cols:] == 55).all(), "wrote past the plan's rows"
        return out[:m * self.cols].reshape(m, self.cols)

    def want(self):
        """(results, bound of each one's error from the fp32 sums)."""
        y = np.zeros((len(self.x), self.N))
        size = np.zeros_like(y)
        for e in range(self.E):
            lo, hi = self.offsets[e], self.offsets[e + 1]
            if lo == hi:
                continue
            w = ref.w4_dequant(self.packed[e], self.scales[e],
                               None if self.zeros is None else self.zeros[e], self.fmt, self.group)
            a = self.x[lo:hi].astype(np.float64)
            y[lo:hi] = a @ w.T
            size[lo:hi] = np.abs(a) @ np.abs(w).T
        size *= 2.0 ** -23 * (self.K / 16 + 64)
        if self.act:
            h = self.N // 2
            # |d SiLU| <= 1.1, so gate errors count 1.1 |up|, up errors |SiLU(gate)|
            s = ref.swiglu(np.concatenate((y[:, :h], np.ones_like(y[:, :h])), 1))
            size = 1.1 * size[:, :h] * np.abs(y[:, h:]) + np.abs(s) * size[:, h:] + size[:, :h] * size[:, h:]
            y = ref.swiglu(y)
        return y, size

    def check(self, out):
        assert self.status.item() == 0
        y, size = self.want()
        assert (np.abs(out - y) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(y) + 1.01 * size + 1e-37).all()
        if y.size >= 64:
            assert np.linalg.norm(out - y) <= (2.0 ** -8 + 2.0 ** -13) * np.linalg.norm(y)


def activations(rows, K, seed):
    rng = np.random.default_rng(seed)
    return ref.bf16_round(rng.normal(size=(rows, K)).astype(np.float32))


FORMATS = [("int4", 32), ("int4", 64), ("int4", 128), ("int4z", 32), ("int4z", 64), ("int4z", 128),
           ("e2m1", 32)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("N,K,counts", [
    (2, 128, [1]), (64, 256, [1, 0, 2]), (130, 384, [8]), (126, 1408, [0, 9, 0, 3]),
    (514, 2048, [1, 1, 1, 1]), (1000, 640, [17, 33, 0, 70]), (4096, 512, [5]),
])
def test_w4_sizes(N, K, counts, fmt, group, act):
    c = Call(activations(sum(counts), K, N), counts, weights(len(counts), N, K, fmt, group, K),
             fmt, group, act)
    c.check(c.run())


@pytest.mark.parametrize("fmt,group", [("int4z", 32), ("e2m1", 32), ("int4", 64)])
@pytest.mark.parametrize("N,K", [(1, 64), (7, 192), (63, 320), (129, 1600), (2049, 64), (257, 14336)])
def test_w4_odd_columns(N, K, fmt, group):
    """An odd N: rows of C start at odd elements; K that ends inside a tile."""
    if fmt != "int4":
        K += 32
    c = Call(activations(6, K, N), [2, 4], weights(2, N, K, fmt, group, N), fmt, group)
    c.check(c.run())


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 65, 129])
def test_w4_row_counts(rows):
    for fmt, group in (("int4", 128), ("e2m1", 32)):
        c = Call(activations(rows, 1024, rows), [0, rows, 0], weights(3, 200, 1024, fmt, group, 1),
                 fmt, group)
        c.check(c.run())


def test_w4_many_experts_mostly_empty():
    rng = np.random.default_rng(2)
    counts = (rng.random(256) < 0.1) * rng.integers(1, 4, 256)
    c = Call(activations(int(counts.sum()), 256, 3), counts, weights(256, 96, 256, "int4", 64, 4),
             "int4", 64)
    c.check(c.run())


def test_w4_no_rows_at_all():
    c = Call(activations(0, 256, 3), [0, 0], weights(2, 64, 256, "int4", 64, 4), "int4", 64, max_rows=8)
    assert c.run().size == 0 and c.status.item() == 0


def test_w4_rows_past_the_plan_are_left_alone():
    c = Call(activations(3, 256, 3), [1, 2], weights(2, 64, 256, "int4", 64, 4), "int4", 64, max_rows=40)
    c.check(c.run())


def test_w4_calls_repeat_bit_for_bit():
    """The same workspace over and over, other calls between, another stream."""
    for shape in ((64, 14336, [3]), (4096, 768, [1, 0, 9]), (300, 4096, [40])):
        N, K, counts = shape
        c = Call(activations(sum(counts), K, N), counts, weights(len(counts), N, K, "int4z", 64, K),
                 "int4z", 64)
        c.check(c.run())
        first = c.bits
        for stream in (None, torch.cuda.Stream(), None):
            c.C.fill_(55.0)
            c.run(stream)
            np.testing.assert_array_equal(first, c.bits)


def test_w4_one_workspace_for_calls_of_other_shapes():
    big = Call(activations(5, 4096, 1), [5], weights(1, 700, 4096, "int4", 128, 1), "int4", 128)
    small = Call(activations(2, 256, 1), [1, 1], weights(2, 40, 256, "e2m1", 32, 1), "e2m1", 32)
    small.args.workspace = big.args.workspace
    for _ in range(3):
        big.check(big.run())
        small.check(small.run())


@pytest.mark.parametrize("act", [False, True])
def test_w4_gathers_the_tokens_of_several_ranks(act):
    """Without A the rows come from the ranks' tokens, as ep_plan orders them."""
    R, T, k, El, N, K = 3, 5, 2, 4, 72, 320
    rng = np.random.default_rng(6)
    ids = np.stack([[rng.permutation(R * El)[:k] for _ in range(T)] for _ in range(R)]).astype(np.int32)
    x = activations(R * (T + 2), K, 8).reshape(R, T + 2, K)  # two spare tokens a rank
    conf = cfg(El, N, K, R, k, T)
    conf.my_rank, conf.max_tokens_per_rank = 1, T + 2
    dev = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    rows = ep.ep_plan_sizes(conf)
    plan = dict(expert_offsets=dev(El + 1), src_info=dev(rows, 2), seg_offsets=dev(El, R + 1),
                send_counts=dev(El, R), gather_idx=dev(rows), m_total=dev(1), status=dev(1))
    ep.ep_plan(conf, torch.from_numpy(ids).cuda(), ep.ep_plan_out(
        **{n: ep.ptr(t) for n, t in plan.items()}, max_rows=rows))
    off = plan["expert_offsets"].cpu().numpy()
    gi = plan["gather_idx"].cpu().numpy()[:off[-1]]
    flat = x[:, :T].reshape(R * T, K)[gi // k]
    c = Call(flat, np.diff(off), weights(El, N, K, "int4z", 32, 9), "int4z", 32, act, max_rows=rows)
    xs = [torch.from_numpy(x[r]).to("cuda", torch.bfloat16) for r in range(R)]
    c.cfg = conf
    c.args.A = 0
    c.args.gather_idx = ep.ptr(plan["gather_idx"])
    for r in range(R):
        c.args.x_ptrs[r] = ep.ptr(xs[r])
    out = c.run()
    c.check(out)
    # an index outside the token tables: that row is skipped, the call says so
    bad = plan["gather_idx"].clone()
    bad[0], bad[1] = R * T * k, -1
    c.args.gather_idx = ep.ptr(bad)
    c.C.fill_(55.0)
    again = c.run()
    assert c.status.item() == ep.EP_STATUS_BOUNDS
    assert (again[:2] == 55).all()
    np.testing.assert_array_equal(again[2:], out[2:])


@pytest.mark.parametrize("offsets", [[0, 3, 9], [0, -1, 4], [2, 4, 1], [0, 5, 4]])
def test_w4_bad_offsets_are_reported(offsets):
    """Offsets that do not rise from within [0, max_rows] to its end: nothing is written."""
    c = Call(activations(4, 256, 3), [2, 2], weights(2, 64, 256, "int4", 64, 4), "int4", 64, max_rows=8)
    c.off.copy_(torch.tensor(offsets, dtype=torch.int32))
    torch.cuda.synchronize()
    ep.ep_matvec_w4(c.cfg, c.args)
    torch.cuda.synchronize()
    assert c.status.item() == ep.EP_STATUS_BOUNDS
    assert (c.C == 55).all()
    c.off.copy_(torch.tensor([0, 2, 4], dtype=torch.int32))
    c.status.zero_()
    c.check(c.run())


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_w4_infinities_and_nan_stay_in_their_rows(fmt, group):
    x = activations(12, 512, 4)
    x[3, 100], x[7, 511], x[8, 0] = np.inf, np.nan, -np.inf
    c = Call(x, [12], weights(1, 100, 512, fmt, group, 4), fmt, group)
    out = c.run()
    clean = [i for i in range(12) if i not in (3, 7, 8)]
    with np.errstate(invalid="ignore"):
        y, size = c.want()
    assert np.isnan(out[7]).all()
    np.testing.assert_array_equal(np.isnan(out[[3, 8]]), np.isnan(y[[3, 8]]))
    np.testing.assert_array_equal(np.sign(out[[3, 8]]), np.sign(y[[3, 8]]))
    assert (np.abs(out - y)[clean] <= 2.0 ** -7.9 * np.abs(y[clean]) + size[clean]).all()


def test_w4_extreme_block_scales():
    """Scale bytes at both ends; a NaN scale makes its weight row's results NaN alone."""
    x = activations(4, 128, 5) * np.float32(2.0 ** -40)
    packed, scales, _ = weights(1, 40, 128, "e2m1", 32, 6)
    scales[0, 0], scales[0, 1], scales[0, 2] = 0, 1, 254
    scales[0, 3, 1] = 255
    c = Call(x, [4], (packed, scales, None), "e2m1", 32)
    out = c.run()
    assert np.isnan(out[:, 3]).all()
    y, size = c.want()
    ok = [n for n in range(40) if n != 3]
    err = np.abs(out - y)[:, ok]
    assert (err <= 2.0 ** -7.9 * np.abs(y[:, ok]) + size[:, ok] + 1e-37).all()


def test_w4_misaligned_output():
    c = Call(activations(9, 256, 3), [4, 5], weights(2, 66, 256, "int4", 64, 4), "int4", 64)
    want = c.run()
    c.C.fill_(55.0)
    c.args.C = ep.ptr(c.C) + 2
    torch.cuda.synchronize()
    ep.ep_matvec_w4(c.cfg, c.args)
    torch.cuda.synchronize()
    out = c.C.float().cpu().numpy()
    np.testing.assert_array_equal(out[1:1 + want.size], want.flatten())
    assert out[0] == 55 and (out[1 + want.size:] == 55).all()


def test_w4_large_offsets():
    """Weights past 2^32 bytes: the last experts' rows, against the same expert alone."""
    E, N, K = 40, 16384, 14336  # 4.7 GB
    W = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    W.random_(0, 256)
    S = torch.full((E, N, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    x = torch.from_numpy(activations(3, K, 1)).to("cuda", torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    for experts, weight in ((E, W), (1, W[E - 1:].clone())):
        conf = cfg(experts, N, K)
        off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        off[experts] = 3
        C = torch.zeros(3, N, dtype=torch.bfloat16, device="cuda")
        n = ep.ep_matvec_w4_sizes(conf)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        a = ep.ep_w4_args(A=ep.ptr(x), W=ep.ptr(weight), w_scales=ep.ptr(S), w_format=ep.EP_W4_INT,
                          group_size=128, expert_offsets=ep.ptr(off), max_rows=3, C=ep.ptr(C),
                          workspace=ep.ptr(ws), workspace_bytes=n, status=ep.ptr(status))
        ep.ep_matvec_w4(conf, a)
        torch.cuda.synchronize()
        outs.append(C.float())
    assert status.item() == 0
    assert torch.equal(outs[0], outs[1])
    w = ref.w4_dequant(W[E - 1, :8].cpu().numpy(), np.full((8, K // 128), float(S[0, 0, 0])), None,
                       "int4", 128)
    y = x.double().cpu().numpy() @ w.T
    np.testing.assert_allclose(outs[0][:, :8].cpu().numpy(), y, rtol=2.0 ** -8, atol=1e-3 * np.abs(y).max())
