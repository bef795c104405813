"""The residual norm and its gradient on the GPU against their formulas in 64 bits."""

import pytest
import torch

import moe_expert_gemm_gb300 as ep
import rows_reference as ref
from rows_reference import BF16, F32

pytestmark = pytest.mark.gpu

ROWS = {torch.float32: ep.EP_ROWS_F32, torch.bfloat16: ep.EP_ROWS_BF16}
STEP = {torch.float32: F32, torch.bfloat16: BF16}
# Relative error of v before its last rounding: the sum of squares passes at most 64 additions in a
# thread and 10 in the block, the mean and eps two, halved by the root (error 4); then the products.
REL = 48 * F32
B, F = torch.bfloat16, torch.float32


def cfg(tokens, n=64):
    return ep.ep_config(1, 0, 1, 1, tokens, max(tokens, 1), 64, n, 2 * n, ep.EP_BF16, -1, 0)


def strided(rows, cols, dtype, gap, gen, scale=1.0):
    """Random rows that lie cols + gap apart, and what lies behind them."""
    base = (scale * torch.randn(rows, cols + gap, generator=gen)).to(dtype).cuda()
    return base[:, :cols], base


def norm_call(x, residual, weight, eps, sum=None, y=None, q=None, s=None, stream=None):
    st = lambda v: 0 if v is None else v.stride(0) if v.shape[0] > 1 else 0
    rt = residual if residual is not None else sum
    a = ep.ep_add_rmsnorm_args(x=ep.ptr(x), x_stride=st(x), residual=ep.ptr(residual),
                               residual_stride=st(residual), residual_dtype=ROWS[rt.dtype] if rt is not None else 0,
                               weight=ep.ptr(weight), weight_dtype=ROWS[weight.dtype], eps=eps,
                               hidden=x.shape[1], sum=ep.ptr(sum), sum_stride=st(sum), y=ep.ptr(y),
                               y_stride=st(y), q=ep.ptr(q), q_scales=ep.ptr(s))
    ep.ep_add_rmsnorm(cfg(x.shape[0]), a, stream)


SHAPES = [(1, 7168, 0), (3, 1, 0), (2, 7, 0), (5, 128, 8), (4, 129, 0), (333, 1111, 3), (64, 4096, 0),
          (1000, 256, 0), (2, 16384, 0), (3, 16383, 1), (5000, 72, 8), (17, 1000, 4)]


@pytest.mark.parametrize("tokens,n,gap", SHAPES)
@pytest.mark.parametrize("stream_type,weight_type", [(None, B), (B, F), (F, B)])
def test_norm(tokens, n, gap, stream_type, weight_type):
    gen = torch.Generator().manual_seed(tokens * 31 + n)
    x, _ = strided(tokens, n, B, gap, gen)
    residual = None if stream_type is None else strided(tokens, n, stream_type, gap, gen, 3.0)[0]
    weight = (1 + 0.3 * torch.randn(n, generator=gen)).to(weight_type).cuda()
    total, behind = strided(tokens, n, stream_type or F, gap, gen)
    kept = behind[:, n:].clone()
    y, y_behind = strided(tokens, n, B, gap, gen)
    y_kept = y_behind[:, n:].clone()
    q = torch.zeros(tokens, n, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(tokens, (n + 127) // 128, device="cuda")
    norm_call(x, residual, weight, 1e-6, total, y, q, s)
    torch.cuda.synchronize()
    h, v = ref.norm(x, residual, weight, 1e-6)
    # (fp32: one rounding in the sum, a second in the type it is stored in)
    assert ((total.double() - h).abs() <= (F32 + STEP[total.dtype]) * h.abs()).all()
    assert ((y.double() - v).abs() <= (BF16 + REL) * v.abs() + 2.0 ** -133).all()
    ref.check_e4m3(q, s, v, REL)
    assert torch.equal(behind[:, n:], kept) and torch.equal(y_behind[:, n:], y_kept)
    # each output alone has the same bits
    y2, q2, s2, total2 = y.clone(), torch.zeros_like(q), torch.zeros_like(s), torch.zeros_like(total)
    norm_call(x, residual, weight, 1e-6, y=y2)
    norm_call(x, residual, weight, 1e-6, q=q2, s=s2)
    norm_call(x, residual, weight, 1e-6, sum=total2)
    assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(total2, total)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("tokens,n", [(1, 64), (300, 4096), (77, 1111)])
def test_in_place(tokens, n):
    gen = torch.Generator().manual_seed(n)
    x, _ = strided(tokens, n, B, 0, gen)
    res, _ = strided(tokens, n, F, 0, gen)
    w = torch.ones(n, device="cuda")
    total, y = torch.zeros_like(res), torch.zeros_like(x)
    norm_call(x, res, w, 1e-5, total, y)
    x2, res2 = x.clone(), res.clone()
    norm_call(x2, res2, w, 1e-5, res2, x2)  # sum over the residual, y over x
    assert torch.equal(res2, total) and torch.equal(x2, y)
    x3, y3 = x.clone(), torch.zeros_like(x)
    norm_call(x3, x.clone(), w, 1e-5, x3, y3)  # sum over x
    both = torch.zeros_like(x)
    norm_call(x, x.clone(), w, 1e-5, both)
    assert torch.equal(x3, both)


def test_addresses_of_single_elements():
    """Rows that start anywhere an element may."""
    n, T = 1024, 9
    gen = torch.Generator().manual_seed(3)
    buf = lambda dtype, off: torch.randn(T * n + 8, generator=gen).cuda().to(dtype)[off:off + T * n].view(T, n)
    x, res, y, total = buf(B, 1), buf(F, 3), buf(B, 5), buf(F, 1)
    w = buf(B, 7)[0]
    q = torch.zeros(T * n + 8, dtype=torch.uint8, device="cuda")[3:3 + T * n].view(T, n)
    s = torch.zeros(T, n // 128, device="cuda")
    norm_call(x, res, w, 1e-6, total, y, q, s)
    h, v = ref.norm(x, res, w, 1e-6)
    assert ((total.double() - h).abs() <= 2 * F32 * h.abs()).all()
    assert ((y.double() - v).abs() <= (BF16 + REL) * v.abs()).all()
    ref.check_e4m3(q.view(torch.float8_e4m3fn), s, v, REL)


@pytest.mark.parametrize("n,pad", [(1024, 0), (1111, 2), (203, 1), (4099, 5)])
@pytest.mark.parametrize("h_type", [B, F])
def test_gradient_addresses_of_single_elements(n, pad, h_type):
    """The gradient's rows, each tensor's at another place behind a 16-byte boundary, with gaps of
    another size each, and over an input."""
    T = 13
    gen = torch.Generator().manual_seed(n)

    def rows(dtype, off, gap):
        base = torch.randn(T * (n + gap) + 8, generator=gen).cuda().to(dtype)
        return base[off:off + T * (n + gap)].view(T, n + gap)[:, :n], base

    h, _ = rows(h_type, 1, pad)
    dy, _ = rows(B, 3, pad + 1)
    dsum, _ = rows(h_type, 2, 0)
    dh, dh_base = rows(h_type, 3, 2 * pad)
    dx, dx_base = rows(B, 7, pad)
    w = rows(F, 1, 0)[0][0]
    before = [b.clone() for b in (dh_base, dx_base)]
    dw = torch.zeros(n, device="cuda")
    back_call(h, dy, w, dsum, dh, dx, dw)
    want, want_w, size, size_w = ref.norm_backward(h, dy, w, dsum, 1e-6)
    off = 256 * F32 * size
    assert ((dh.double() - want).abs() <= STEP[h_type] * (want.abs() + off) + off).all()
    assert ((dx.double() - want).abs() <= BF16 * (want.abs() + off) + off).all()
    assert ((dw.double() - want_w).abs() <= 128 * F32 * size_w).all()
    for base, old, view, gap, at in ((dh_base, before[0], dh, 2 * pad, 3), (dx_base, before[1], dx, pad, 7)):
        outside = torch.ones_like(base, dtype=torch.bool)
        outside[at:at + T * (n + gap)].view(T, n + gap)[:, :n] = False
        assert torch.equal(base[outside], old[outside])
    over = dsum.clone() if dsum.is_contiguous() else dsum
    moved = rows(h_type, 2, 0)[0]
    moved.copy_(over)
    back_call(h, dy, w, moved, moved)
    assert torch.equal(moved, dh)


def test_zeros_infinities_and_nan():
    n, T = 640, 6
    x = torch.randn(T, n, generator=torch.Generator().manual_seed(0)).cuda().to(B)
    x[1] = 0
    x[2, 17] = torch.nan
    x[3, 300] = torch.inf
    x[4, 5], x[4, 6] = torch.inf, -torch.inf
    w = torch.ones(n, device="cuda")
    w[130] = torch.inf  # of a group of its own
    y = torch.zeros_like(x)
    q = torch.zeros(T, n, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.zeros(T, n // 128, device="cuda")
    norm_call(x, None, w, 1e-6, y=y, q=q, s=s)
    _, v = ref.norm(x, None, w, 1e-6)
    for t in (0, 1, 5):
        fine = v[t].isfinite()
        assert ((y[t].double() - v[t]).abs()[fine] <= (BF16 + REL) * v[t].abs()[fine]).all()
        assert torch.equal(y[t].double()[~fine].nan_to_num(7, 8, 9), v[t][~fine].nan_to_num(7, 8, 9))
    assert y[2].isnan().all()
    assert y[3, 300].isnan() and (y[3, :130] == 0).all()  # r is 0 there
    assert y[4, 5].isnan()
    ref.check_e4m3(q, s, v, REL)
    assert s[0, 1].isnan() and s[0, 0].isfinite()
    assert (s[1, 0] == ref.TINY) and (q[1, :128].float() == 0).all()


def test_eps_of_zero_and_tiny_rows():
    x = torch.full((2, 256), 2.0 ** -60, device="cuda", dtype=B)
    x[1] = 0
    w, y = torch.ones(256, device="cuda"), torch.zeros(2, 256, device="cuda", dtype=B)
    norm_call(x, None, w, 0.0, y=y)
    assert (y[0] == 1).all() and y[1].isnan().all()


def back_call(h, dy, weight, dsum=None, dh=None, dx=None, dweight=None, eps=1e-6, stream=None):
    st = lambda v: 0 if v is None else v.stride(0) if v.shape[0] > 1 else 0
    c = cfg(h.shape[0])
    size = ep.ep_add_rmsnorm_backward_sizes(c, h.shape[1])
    work = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, of any contents
    a = ep.ep_add_rmsnorm_backward_args(h=ep.ptr(h), h_stride=st(h), h_dtype=ROWS[h.dtype], dy=ep.ptr(dy),
                                        dy_stride=st(dy), dsum=ep.ptr(dsum), dsum_stride=st(dsum),
                                        weight=ep.ptr(weight), weight_dtype=ROWS[weight.dtype], eps=eps,
                                        hidden=h.shape[1], dh=ep.ptr(dh), dh_stride=st(dh), dx=ep.ptr(dx),
                                        dx_stride=st(dx), dweight=ep.ptr(dweight), workspace=ep.ptr(work),
                                        workspace_bytes=size)
    ep.ep_add_rmsnorm_backward(c, a, stream)
    return work


@pytest.mark.parametrize("tokens,n,gap", SHAPES + [(8192, 512, 0), (3001, 264, 0)])
@pytest.mark.parametrize("h_type,weight_type,through", [(B, F, True), (F, B, True), (B, B, False)])
def test_norm_backward(tokens, n, gap, h_type, weight_type, through):
    gen = torch.Generator().manual_seed(tokens * 7 + n)
    h, _ = strided(tokens, n, h_type, gap, gen, 3.0)
    dy, _ = strided(tokens, n, B, gap, gen)
    dsum = strided(tokens, n, h_type, gap, gen)[0] if through else None
    weight = (1 + 0.3 * torch.randn(n, generator=gen)).to(weight_type).cuda()
    dh, behind = strided(tokens, n, h_type, gap, gen)
    kept = behind[:, n:].clone()
    dx, _ = strided(tokens, n, B, gap, gen)
    dweight = torch.full((n,), torch.nan, device="cuda")
    work = back_call(h, dy, weight, dsum, dh, dx, dweight)
    torch.cuda.synchronize()
    want, want_w, size, size_w = ref.norm_backward(h, dy, weight, dsum, 1e-6)
    # sums of n values: at most 64 in a thread, 10 in the block; r (48, as above) enters three times
    off = 256 * F32 * size
    assert ((dh.double() - want).abs() <= STEP[h_type] * (want.abs() + off) + off).all()
    assert ((dx.double() - want).abs() <= BF16 * (want.abs() + off) + off).all()
    # at most tokens additions one after the other, in whatever order, and r
    assert ((dweight.double() - want_w).abs() <= (min(tokens, 1024) + 64) * F32 * size_w).all()
    assert torch.equal(behind[:, n:], kept)
    # alone, in place, and again: the same bits
    dh2, dx2, dw2 = torch.zeros_like(dh), dy.clone(), torch.zeros_like(dweight)
    back_call(h, dy, weight, dsum, dh2)
    back_call(h, dx2, weight, dsum, None, dx2)
    back_call(h, dy, weight, dsum, None, None, dw2)
    assert torch.equal(dh2, dh) and torch.equal(dx2, dx) and torch.equal(dw2, dweight)
    own = h.clone()
    back_call(own, dy, weight, dsum, own)
    assert torch.equal(own, dh)
    if through:
        over = dsum.clone()
        back_call(h, dy, weight, over, over)
        assert torch.equal(over, dh)
    del work


def test_gradient_against_differences():
    """The gradients of the forward kernel's own v, by differences of it (fp32 stream, so that a
    step of h is no rounding; v read back in 8 + 16 bits would be too coarse: from the formula in 64
    bits, which the forward test holds the kernel to)."""
    gen = torch.Generator().manual_seed(11)
    T, n = 5, 96
    h = torch.randn(T, n, generator=gen).cuda()
    dy = torch.randn(T, n, generator=gen).cuda().to(B)
    w = torch.randn(n, generator=gen).cuda()
    dh, dw = torch.zeros_like(h), torch.zeros(n, device="cuda")
    back_call(h, dy, w, dh=dh, dweight=dw, eps=0.1)
    value = lambda h, w: (ref.norm(h, None, w, 0.1)[1] * dy.double()).sum()
    step = 2.0 ** -12
    for i in range(n):
        for t in range(T):
            d = torch.zeros(T, n, dtype=torch.float64, device="cuda")
            d[t, i] = step
            slope = (value(h.double() + d, w) - value(h.double() - d, w)) / (2 * step)
            assert abs(float(slope - dh[t, i])) < 2e-5  # third derivatives of size ~10 by step^2, and fp32
        d = torch.zeros(n, dtype=torch.float64, device="cuda")
        d[i] = step
        slope = (value(h, w.double() + d) - value(h, w.double() - d)) / (2 * step)
        assert abs(float(slope - dw[i])) < 2e-5


def test_gradients_of_no_tokens():
    dw = torch.ones(64, device="cuda")
    a = ep.ep_add_rmsnorm_backward_args(hidden=64, eps=1e-6, dweight=ep.ptr(dw))
    ep.ep_add_rmsnorm_backward(cfg(0), a)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_past_31_bits():
    """The last rows of a batch of more than 2^31 elements."""
    n, T = 16384, 131072 + 40
    x = torch.zeros(T, n, dtype=B, device="cuda")
    x[-3:] = torch.randn(3, n, generator=torch.Generator().manual_seed(1)).cuda().to(B)
    w, y = torch.ones(n, device="cuda"), torch.empty(T, n, dtype=B, device="cuda")
    norm_call(x, None, w, 1e-6, y=y)
    _, v = ref.norm(x[-3:], None, w, 1e-6)
    assert ((y[-3:].double() - v).abs() <= (BF16 + REL) * v.abs()).all() and (y[:-3] == 0).all()
    dw, dh = torch.zeros(n, device="cuda"), y
    back_call(x, x, w, dh=dh, dweight=dw)
    want, want_w, size, size_w = ref.norm_backward(x[-3:], x[-3:], w, None, 1e-6)
    off = 256 * F32 * size
    assert ((dh[-3:].double() - want).abs() <= BF16 * (want.abs() + off) + off).all()
    assert ((dw.double() - want_w).abs() <= 100 * F32 * size_w).all()
