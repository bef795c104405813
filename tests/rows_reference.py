"""The residual norm, its gradient, rows in 8 bits and the layer of a few tokens in 64 bits, written
from their definitions (include/moe_ep.h), for the tests to compare with. Tensors on any device."""

import torch

BF16, F32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4  # half a step, relative to the value
TINY = 2.0 ** -126  # smallest scale of a group


def norm(x, residual, weight, eps):
    """(h, v) of rows."""
    h = x.double() if residual is None else x.double() + residual.double()
    return h, h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps) * weight.double()


def norm_backward(h, dy, weight, dsum, eps):
    """(dh, dweight, and the magnitudes that each is summed from)."""
    h, dy, w = h.double(), dy.double(), weight.double()
    n = h.shape[-1]
    r = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    g = dy * w
    dh = r * (g - h * r * r * (g * h).sum(-1, keepdim=True) / n)
    size = r * (g.abs() + h.abs() * r * r * (g * h).abs().sum(-1, keepdim=True) / n)
    if dsum is not None:
        dh, size = dh + dsum.double(), size + dsum.double().abs()
    return dh, (dy * h * r).sum(0), size, (dy * h * r).abs().sum(0)


def groups(v, n=128):
    """[..., cols] -> [..., ceil(cols / n), n], zeros past the end."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % n)).unflatten(-1, (-1, n))


def scales(v):
    """Scale of each 128 columns; NaN where one of them is not finite."""
    s = (groups(v).abs().amax(-1) / 448).clamp(min=TINY)
    return torch.where(groups(v).isfinite().all(-1), s, torch.nan)


def e4m3_nearest(v):
    """Nearest e4m3 numbers (as doubles), ties to even."""
    a = v.abs().clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step)


def requantised(v):
    """Rows as their codes and scales stand for them."""
    s = scales(v)
    return (e4m3_nearest(groups(v) / s[..., None]) * s[..., None]).flatten(-2)[..., :v.shape[-1]]


def wide(q, s):
    """Values of [..., rows][cols] e4m3 codes with scales [..., rows][ceil(cols/128)]."""
    return (groups(q.double()) * s.double()[..., None]).flatten(-2)[..., :q.shape[-1]]


def wide_blocks(q, s):
    """Values of [..., rows][cols] codes with the scales of 128 x 128 blocks."""
    return q.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


def check_e4m3(q, s, v, rel):
    """Codes q [rows][cols] and scales s of values v that may be off by rel: scales near, codes the
    nearest, groups with something not finite NaN as a whole."""
    want = scales(v)
    bad = want.isnan()
    assert torch.equal(s.isnan(), bad)
    assert ((s.double() - want).abs()[~bad] <= (rel + 2 * F32) * want[~bad]).all()
    q = groups(q.double())  # (zeros past a row's end)
    if bad.any():
        there = groups(torch.ones_like(v)).bool()
        assert q[bad][there[bad]].isnan().all()
    # a code is off by half a step of a normal number, or of the subnormals' 2^-9
    off = (q * s.double()[..., None] - groups(v)).abs()[~bad]
    s, v = s.double()[~bad][:, None], groups(v)[~bad].abs()
    assert (off <= (E4M3 + rel + 4 * F32) * v + 2.0 ** -10 * s).all()


def swiglu(g):
    """SiLU(gate) * up of [..., 2I]."""
    gate, up = g.double().chunk(2, -1)
    return gate * torch.sigmoid(gate) * up


def layer_few(x, ids, gates, W1, W2, first, fp8):
    """(out, and a bound of what sums in fp32 and the roundings in between may change): x, W1, W2
    as values in 64 bits; ids global, this rank's experts from `first` on."""
    T, H = x.shape
    E, I = W1.shape[0], W1.shape[1] // 2
    out, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    x, W1, W2, gates, ids = (v.cpu() for v in (x, W1, W2, gates.double(), ids))
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j]) - first
            if not 0 <= e < E:
                continue
            gu = W1[e] @ x[t]
            # n values sum in fp32 to within n half steps of the sum of their sizes
            err = (H + 8) * F32 * (W1[e].abs() @ x[t].abs())
            a = swiglu(gu)
            silu = (gu[:I] * torch.sigmoid(gu[:I])).abs()
            # |SiLU'| <= 1.1
            ea = 1.1 * err[:I] * (gu[I:].abs() + err[I:]) + silu * err[I:] + 16 * F32 * a.abs()
            if fp8:
                rounded = requantised(a[None])[0]
                ea = ea + E4M3 * (a.abs() + ea) + 2.0 ** -10 * scales(a[None])[0].repeat_interleave(128)[:I]
            else:
                rounded = a.bfloat16().double()
                ea = ea + BF16 * (a.abs() + ea)
            g = gates[t, j]
            out[t] += g * (W2[e] @ rounded)
            # (the reference rounds too: both may be on either side)
            bound[t] += g.abs() * (W2[e].abs() @ (2 * ea) + (I + 8) * F32 * (W2[e].abs() @ (a.abs() + ea)))
    return out, bound + (ids.shape[1] + 2) * F32 * out.abs()
