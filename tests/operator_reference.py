"""The router, the combine's gradient and the 4-bit products in plain numpy, 64 bits,
written from their definitions (include/moe_ep.h), for the tests to compare with."""

import numpy as np

LOWEST = {"f32": -float(np.finfo(np.float32).max), "bf16": -3.3895313892515355e38}


def bf16_round(x):
    """fp32 -> nearest bf16 (ties to even), as fp32; NaN stays NaN."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((b.astype(np.uint64) + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return np.where(np.isnan(x), np.float32(np.nan), r.view(np.float32))


def scores(l, masked, score):
    """Scores of one token's logits (masked: 0); NaN-free."""
    l = np.where(masked, 0.0, l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(masked, 0.0, 1 / (1 + np.exp(-l)))
    if masked.all():
        return np.zeros_like(l)
    with np.errstate(under="ignore"):
        e = np.where(masked, 0.0, np.exp(l - l[~masked].max()))
    return e / e.sum()


def choice_values(l, masked, score, bias):
    """Choice value of every expert (masked: -inf)."""
    v = l if bias is None else scores(l, masked, score) + bias
    return np.where(masked, -np.inf, v)


def group_worth(l, masked, score, bias, n_groups, group_top):
    v = choice_values(l, masked, score, bias)
    if group_top == 2 and bias is None:
        v = np.where(masked, -np.inf, scores(l, masked, score))
    worth = np.full(n_groups, -np.inf)
    for g, part in enumerate(v.reshape(n_groups, -1)):
        best = np.sort(part[~masked.reshape(n_groups, -1)[g]])[::-1][:group_top]
        if best.size:
            worth[g] = best.sum()
    return worth


def chosen(l, masked, score, bias, k, n_groups=1, topk_groups=1, group_top=1):
    """The top_k experts of one token."""
    E = l.size
    member = np.ones(E, bool)
    if topk_groups < n_groups:
        worth = group_worth(l, masked, score, bias, n_groups, group_top)
        keep = sorted(range(n_groups), key=lambda g: (-worth[g], g))[:topk_groups]
        member = np.isin(np.arange(E) // (E // n_groups), keep)
    v = choice_values(l, masked, score, bias)
    order = sorted(np.nonzero(member)[0], key=lambda i: (bool(masked[i]), -v[i], i))
    return np.array(order[:k])


def gates_of(l, ids, score, renorm, scale, lowest):
    """The gates of the chosen experts of one token."""
    if np.isnan(l).any() or (score == "softmax" and np.isposinf(l).any()):
        return np.full(len(ids), np.nan)
    masked = l <= lowest
    if score == "softmax" and renorm:
        a = scores(l[ids], masked[ids], score)
    else:
        a = scores(l, masked, score)[ids]
        if renorm and a.sum() > 0:
            a = a / a.sum()
    return a * scale


def gates_backward(l, ids, dg, score, renorm, scale, lowest):
    """(dlogits of one token, the magnitude each is summed from)."""
    masked = l <= lowest
    d, size = np.zeros_like(l), np.zeros_like(l)
    dg = np.where(masked[ids], 0.0, dg)
    if score == "softmax" and not renorm:
        p = scores(l, masked, score)
        part = dg * p[ids]
        d -= p * part.sum()
        size += p * np.abs(part).sum()
        d[ids] += part
        size[ids] += np.abs(part)
    else:
        if score == "softmax":
            a, slope = scores(l[ids], masked[ids], score), 1.0
        else:
            a = scores(l[ids], masked[ids], score)
            slope = scores(-l[ids], masked[ids], score)
        c, size_c = 0.0, 0.0
        if renorm:
            a = a / a.sum() if a.sum() > 0 else a * 0
            c, size_c = (dg * a).sum(), np.abs(dg * a).sum()
        d[ids] = a * slope * (dg - c)
        size[ids] = a * slope * (np.abs(dg) + size_c)
    return d * scale, size * scale


E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def w4_dequant(packed, scales, zeros, fmt, group):
    """[..., K/2] bytes -> [..., K] values; scales as numbers (e2m1: exponent bytes)."""
    q = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    if fmt == "e2m1":
        s = np.exp2(scales.astype(np.float64) - 127)
        s[scales == 255] = np.nan
        v = E2M1[q]
    else:
        s = scales.astype(np.float64)
        z = np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64)
        v = q - np.repeat(z, group, -1)
    return v * np.repeat(s, group, -1)


def swiglu(y):
    half = y.shape[-1] // 2
    gate, up = y[..., :half], y[..., half:]
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up
