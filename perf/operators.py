"""Cases of the routing and 4-bit expert operators: ep_route, ep_route_backward,
ep_combine_backward and ep_matvec_w4, each in a plain form (elementary torch
operations in 32 bits, rounded once) and as a user calls it (``own``).

Conventions of the framework: E experts, T tokens, top_k experts per token; expert
rows are in plan order (by expert, then token, then slot), ``expert_offsets`` holds
each expert's first row and ``gather_idx`` each row's flat (token, slot) index.
"""

import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# value of each e2m1 code
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one decoded token through a router of 256 experts in 8 groups: pure latency
        dict(name="route one token of 256", op="route", tokens=1, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5, dtype="f32", masked=0),
        # a prefill batch of the 8-expert top-2 layer, router logits in bf16 (many ties)
        dict(name="route 4096 of 8", op="route", tokens=4096, experts=8, top_k=2,
             score="softmax", bias=False, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0, dtype="bf16", masked=0),
        # the whole expert-parallel group's prefill: 8 ranks x 8192 tokens, 256 experts
        dict(name="route 65536 of 256", op="route", tokens=65536, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5, dtype="f32", masked=0),
        # one rank's training batch of the 128-expert layer, gates a softmax of the chosen
        dict(name="route backward 2048 of 128", op="route_backward", tokens=2048, experts=128,
             top_k=8, score="softmax", renorm=True, scale=1.0, dtype="bf16", masked=0),
        # gates that are not renormalised: the gradient reaches every expert's logit
        dict(name="route backward 65536 of 256", op="route_backward", tokens=65536, experts=256,
             top_k=8, score="softmax", renorm=False, scale=1.0, dtype="f32", masked=0),
        # the decode batch's rows: a small fine-tuning step
        dict(name="combine backward 128x8", op="combine_backward", tokens=128, top_k=8, N=7168),
        # one rank's prefill of 8192 tokens, top-8 rows of 7168: the largest call
        dict(name="combine backward 8192x8", op="combine_backward", tokens=8192, top_k=8, N=7168),
        # one decoded token, the up/gate projection of its 8 of 32 experts with the activation
        dict(name="w4 up one token", op="w4", tokens=1, experts=32, top_k=8, K=7168, N=4096,
             format="int4", group=128, act=True),
        # one decoded token, the down projection of 8 of 16 small experts: latency counts
        dict(name="w4 down one token", op="w4", tokens=1, experts=16, top_k=8, K=1536, N=4096,
             format="e2m1", group=32, act=False),
        # one matrix with a long K and zero points (a shared expert), a few tokens
        dict(name="w4 shared 5 tokens", op="w4", tokens=5, experts=1, top_k=1, K=14336, N=4096,
             format="int4z", group=128, act=False),
        # ragged sizes: K and N that end inside a tile, small groups with zero points
        dict(name="w4 ragged 11 tokens", op="w4", tokens=11, experts=12, top_k=3, K=1504, N=2050,
             format="int4z", group=32, act=False),
        # the decode batch of an expert-parallel rank: about 32 rows for each of 32 experts
        dict(name="w4 down 128 tokens", op="w4", tokens=128, experts=32, top_k=8, K=2048, N=7168,
             format="e2m1", group=32, act=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _but(v, step):
    return v + step if v == 3072 else v  # a size that stands for nothing here


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "combine_backward", "w4", "w4"])
    if op == "route":
        tokens = _but(_log(rng, 1, 65536), 1)
        sigmoid = rng.random() < 0.5
        if rng.random() < 0.4:  # groups of equal size
            groups = rng.choice([2, 4, 8])
            per = rng.randint(4, 256 // groups)
            topk_groups = rng.randint(1, groups)
            experts, top_k = groups * per, rng.randint(1, min(8, topk_groups * per))
            group_top = rng.choice([1, 2])
        else:
            groups = topk_groups = group_top = 1
            experts = _log(rng, 8, 256)
            top_k = rng.randint(1, 8)
        # a balance bias goes with sigmoid scores; padded experts are masked
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k,
                    score="sigmoid" if sigmoid else "softmax",
                    bias=sigmoid and rng.random() < 0.7, groups=groups, topk_groups=topk_groups,
                    group_top=group_top, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.choice([0, 0, 1, 5]))
    if op == "route_backward":
        return dict(op=op, tokens=_but(_log(rng, 1, 65536), 1), experts=_log(rng, 8, 256),
                    top_k=rng.randint(1, 8), score=rng.choice(["sigmoid", "softmax"]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0, 0, 1, 5]))
    if op == "combine_backward":
        top_k, N = rng.randint(1, 8), _but(8 * _log(rng, 16, 896), 8)
        return dict(op=op, tokens=_but(_log(rng, 1, 8192), 1), top_k=top_k, N=N)
    fmt = rng.choice(["int4", "int4z", "e2m1"])
    group = 32 if fmt == "e2m1" else rng.choice([32, 64, 128])
    act = rng.random() < 0.5
    experts = rng.choice([1, 4, 8, 12, 16, 32])
    K = _but(group * max(1, _log(rng, 512, 14336) // group), group)
    most = 32 * 2048 * 7168 // (experts * K)  # weights of the largest listed case
    N = _but(max(64, min(_log(rng, 512, 8192), most)), 2)
    if act:  # gate and up rows
        N = 2 * _but(N // 2, 1)
    return dict(op=op, tokens=_log(rng, 1, 128), experts=experts,
                top_k=rng.randint(1, min(8, experts)), K=K, N=N, format=fmt, group=group, act=act)


# ------------------------------------------------------------------ inputs


def _logits(case, g, dev):
    """Router logits: tokens' own preferences plus a popularity of each expert, some
    trailing experts (padding) masked."""
    T, E = case["tokens"], case["experts"]
    l = torch.randn(T, E, generator=g, device=dev)
    l += 0.5 * torch.randn(E, generator=g, device=dev)
    if case["masked"]:
        l[:, E - min(case["masked"], E // 4):] = -math.inf
    return l.to(_DTYPES[case["dtype"]])


def _distinct(T, E, k, g, dev):
    """k distinct experts of each token, in random order."""
    return torch.rand(T, E, generator=g, device=dev).argsort(dim=1)[:, :k].to(torch.int32).contiguous()


def _weights(case, g, dev):
    """4-bit weights of N(0, 1/K) values: two codes a byte (low nibble the even k), the
    scales (and zero points) of groups along k."""
    E, N, K, G = case["experts"], case["N"], case["K"], case["group"]
    packed = torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev)
    e2m1 = case["format"] == "e2m1"
    scales = torch.empty(E, N, K // G, dtype=torch.uint8 if e2m1 else torch.bfloat16, device=dev)
    zeros = torch.empty(E, N, K // G, dtype=torch.uint8, device=dev) if case["format"] == "int4z" else None
    for e in range(E):
        w = torch.randn(N, K // G, G, generator=g, device=dev) / math.sqrt(K)
        if e2m1:
            ex = torch.ceil(torch.log2(w.abs().amax(-1) / 6)).clamp(-100, 100)
            scales[e] = (ex + 127).to(torch.uint8)
            mag = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
            v = w * torch.exp2(-ex)[..., None]
            q = torch.bucketize(v.abs(), mag) + 8 * (v < 0)
        elif zeros is not None:
            lo, hi = w.amin(-1), w.amax(-1)
            s = ((hi - lo) / 15).to(torch.bfloat16)
            z = torch.round(-lo / s.float()).clamp(0, 15)
            scales[e], zeros[e] = s, z.to(torch.uint8)
            q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp(0, 15)
        else:
            s = (w.abs().amax(-1) / 7).to(torch.bfloat16)
            scales[e] = s
            q = (torch.round(w / s.float()[..., None]) + 8).clamp(0, 15)
        q = q.to(torch.uint8).view(N, K // 2, 2)
        packed[e] = q[..., 0] | (q[..., 1] << 4)
    return packed, scales, zeros


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, T = case["op"], case["tokens"]
    s = dict(case=case)
    if op in ("route", "route_backward"):
        E, k = case["experts"], case["top_k"]
        s["logits"] = _logits(case, g, dev)
        if op == "route":
            s["bias"] = 0.1 * torch.randn(E, generator=g, device=dev) if case["bias"] else None
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
            s["gates"] = torch.empty(T, k, device=dev)
        else:
            s["ids"] = _distinct(T, E, k, g, dev)
            s["dgates"] = torch.randn(T, k, generator=g, device=dev)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op == "combine_backward":
        k, N = case["top_k"], case["N"]
        s["rows"] = torch.randn(T, k, N, generator=g, device=dev, dtype=torch.bfloat16)
        s["dout"] = 0.1 * torch.randn(T, N, generator=g, device=dev, dtype=torch.bfloat16)
        s["gates"] = torch.softmax(torch.randn(T, k, generator=g, device=dev), -1)
        s["dgates"] = torch.empty(T, k, device=dev)
        s["drows"] = torch.empty_like(s["rows"])
    else:
        E, k, K, N = case["experts"], case["top_k"], case["K"], case["N"]
        ids = _distinct(T, E, k, g, dev).view(-1).long()
        # the plan: rows by expert, then token, then slot
        gather = torch.argsort(ids, stable=True)
        s["gather_idx"] = gather.to(torch.int32)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        s["offsets"][1:] = torch.cumsum(torch.bincount(ids, minlength=E), 0)
        # the tokens; a few channels carry larger values, as hidden states do
        x = torch.randn(T, K, generator=g, device=dev)
        x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device=dev)] *= 8
        x = x.to(torch.bfloat16)
        # the up/gate projection reads the tokens through the plan, the down projection
        # rows that lie in plan order
        s["x"] = x if case["act"] else x[gather // k].contiguous()
        s["W"], s["scales"], s["zeros"] = _weights(case, g, dev)
        s["C"] = torch.empty(T * k, N // 2 if case["act"] else N, dtype=torch.bfloat16, device=dev)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:
        _handle(s)
    return s


def _handle(s):
    """The argument blocks a program keeps for its calls: pointers and sizes only."""
    import moe_expert_gemm_gb300 as ep

    case, op, T = s["case"], s["case"]["op"], s["case"]["tokens"]
    N = case.get("N", 64)
    cfg = ep.ep_config(n_ranks=1, my_rank=0, n_local_experts=case.get("experts", case["top_k"]),
                       top_k=case["top_k"], num_tokens=T, max_tokens_per_rank=T,
                       K=case.get("K", 64), N=N, msg_bytes=2 * N, dtype=ep.EP_BF16,
                       send_warps=-1, signal_mode=0)
    score = {"sigmoid": ep.EP_SCORE_SIGMOID, "softmax": ep.EP_SCORE_SOFTMAX}
    dtype = {"f32": ep.EP_LOGITS_F32, "bf16": ep.EP_LOGITS_BF16}
    if op == "route":
        a = ep.ep_route_args(logits=ep.ptr(s["logits"]), logits_dtype=dtype[case["dtype"]],
                             score=score[case["score"]], bias=ep.ptr(s["bias"]),
                             n_groups=case["groups"], topk_groups=case["topk_groups"],
                             group_top=case["group_top"], renormalize=int(case["renorm"]),
                             scale=case["scale"], topk_ids=ep.ptr(s["ids"]), gates=ep.ptr(s["gates"]))
    elif op == "route_backward":
        s["status"] = torch.zeros(1, dtype=torch.int32, device=s["logits"].device)
        a = ep.ep_route_backward_args(logits=ep.ptr(s["logits"]), logits_dtype=dtype[case["dtype"]],
                                      score=score[case["score"]], renormalize=int(case["renorm"]),
                                      scale=case["scale"], topk_ids=ep.ptr(s["ids"]),
                                      dgates=ep.ptr(s["dgates"]), dlogits=ep.ptr(s["dlogits"]),
                                      status=ep.ptr(s["status"]))
    elif op == "combine_backward":
        a = ep.ep_combine_backward_args(recv_buf=ep.ptr(s["rows"]), gates=ep.ptr(s["gates"]),
                                        dout=ep.ptr(s["dout"]), dgates=ep.ptr(s["dgates"]),
                                        drows=ep.ptr(s["drows"]))
    else:
        a = ep.ep_w4_args(W=ep.ptr(s["W"]), w_scales=ep.ptr(s["scales"]), w_zeros=ep.ptr(s["zeros"]),
                          w_format=ep.EP_W4_E2M1 if case["format"] == "e2m1" else ep.EP_W4_INT,
                          group_size=case["group"], expert_offsets=ep.ptr(s["offsets"]),
                          max_rows=T * case["top_k"],
                          local_activation=ep.EP_ACT_SWIGLU if case["act"] else ep.EP_ACT_NONE,
                          C=ep.ptr(s["C"]), status=ep.ptr(s["status"]))
        if case["act"]:
            a.x_ptrs[0], a.gather_idx = ep.ptr(s["x"]), ep.ptr(s["gather_idx"])
        else:
            a.A = ep.ptr(s["x"])
        # zero before the first call; every call leaves it ready for the next
        size = ep.ep_matvec_w4_sizes(cfg)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=s["x"].device)
        a.workspace, a.workspace_bytes = ep.ptr(s["workspace"]), size
    s["ep"], s["cfg"], s["args"] = ep, cfg, a


# --------------------------------------------------------------- plain form


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_route(s):
    c, raw = s["case"], s["logits"]
    T, E, k, n = c["tokens"], c["experts"], c["top_k"], c["groups"]
    masked = raw <= torch.finfo(raw.dtype).min
    l = raw.float().masked_fill(masked, -math.inf)
    if c["score"] == "sigmoid":
        u = score = _sigmoid(l)
    else:
        top = l.amax(-1, keepdim=True)
        u = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        score = u / u.sum(-1, keepdim=True)
    v = l if s["bias"] is None else (score + s["bias"]).masked_fill(masked, -math.inf)
    idx = torch.arange(E, device=l.device).expand(T, E)
    if n > 1:
        if c["group_top"] == 1:
            worth = v.view(T, n, -1).amax(-1)
        else:
            # the two best of each group, masked members left out of the sum
            w = (u if s["bias"] is None else v).masked_fill(masked, -math.inf)
            two = w.view(T, n, -1).sort(dim=-1, descending=True).values[..., :2]
            worth = two[..., 0] + torch.where(two[..., 1] == -math.inf, 0.0, two[..., 1])
        best = worth.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        best = best.sort(-1).values
        idx = (best[..., None] * (E // n) + torch.arange(E // n, device=l.device)).view(T, -1)
    order = v.gather(1, idx).sort(dim=-1, descending=True, stable=True).indices[:, :k]
    ids = idx.gather(1, order)
    if c["score"] == "softmax" and c["renorm"]:
        sel = l.gather(1, ids)
        top = sel.amax(-1, keepdim=True)
        a = torch.exp(sel - torch.where(top == -math.inf, torch.zeros_like(top), top))
    else:
        a = score.gather(1, ids).masked_fill(masked.gather(1, ids), 0.0)
    if c["renorm"]:
        total = a.sum(-1, keepdim=True)
        a = torch.where(total == 0, torch.zeros_like(a), a / total)
    return ids.to(torch.int32), a * c["scale"]


def _plain_route_backward(s):
    c, raw = s["case"], s["logits"]
    ids, dg = s["ids"].long(), s["dgates"]
    masked = raw <= torch.finfo(raw.dtype).min
    l = raw.float().masked_fill(masked, -math.inf)
    dl = torch.zeros_like(l)
    if c["score"] == "softmax" and not c["renorm"]:
        top = l.amax(-1, keepdim=True)
        e = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        p = e / e.sum(-1, keepdim=True)
        part = dg * p.gather(1, ids)
        dl = -p * part.sum(-1, keepdim=True)
        dl.scatter_add_(1, ids, part)
    else:
        sel = l.gather(1, ids)
        if c["score"] == "softmax":
            top = sel.amax(-1, keepdim=True)
            a = torch.exp(sel - torch.where(top == -math.inf, torch.zeros_like(top), top))
            slope = torch.ones_like(a)
        else:
            a, slope = _sigmoid(sel), _sigmoid(-sel)
        if c["renorm"]:
            total = a.sum(-1, keepdim=True)
            a = torch.where(total == 0, torch.zeros_like(a), a / total)
            dg = dg - (dg * a).sum(-1, keepdim=True)
        dl.scatter_(1, ids, torch.where(a == 0, torch.zeros_like(a), a * slope * dg))
    return (dl * c["scale"]).to(raw.dtype)


def _plain_combine_backward(s):
    dout = s["dout"].float()[:, None, :]
    dgates = (s["rows"].float() * dout).sum(-1)
    return dgates, (s["gates"][..., None] * dout).to(torch.bfloat16)


def _plain_w4(s):
    c = s["case"]
    T, E, k, K, N, G = c["tokens"], c["experts"], c["top_k"], c["K"], c["N"], c["group"]
    q = torch.stack((s["W"] & 15, s["W"] >> 4), -1).view(E, N, K // G, G)
    if c["format"] == "e2m1":
        scale = (s["scales"].int() << 23).view(torch.float32)  # 2^(code - 127)
        w = torch.tensor(_E2M1, device=q.device)[q.int()]
    else:
        scale = s["scales"].float()
        w = q.float() - (8.0 if s["zeros"] is None else s["zeros"].float()[..., None])
    w = (w * scale[..., None]).view(E, N, K)
    rows = torch.arange(T * k, device=q.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), rows, right=True)
    x = (s["x"][s["gather_idx"].long() // k] if c["act"] else s["x"]).float()
    # every expert's rows in a block of T rows (an expert has at most one of each token)
    place = expert * T + rows - s["offsets"].long()[expert]
    blocks = torch.zeros(E * T, K, device=q.device).index_copy_(0, place, x).view(E, T, K)
    y = torch.bmm(blocks, w.transpose(1, 2)).view(E * T, N)[place]
    if c["act"]:
        gate, up = y[:, :N // 2], y[:, N // 2:]
        y = gate * _sigmoid(gate) * up
    return y.to(torch.bfloat16)


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward,
          "combine_backward": _plain_combine_backward, "w4": _plain_w4}


def run(state):
    op = state["case"]["op"]
    if not own:
        return _PLAIN[op](state)
    ep, stream = state["ep"], torch.cuda.current_stream()
    if op == "route":
        ep.ep_route(state["cfg"], state["args"], stream)
        return state["ids"], state["gates"]
    if op == "route_backward":
        ep.ep_route_backward(state["cfg"], state["args"], stream)
        return state["dlogits"]
    if op == "combine_backward":
        ep.ep_combine_backward(state["cfg"], state["args"], stream)
        return state["dgates"], state["drows"]
    ep.ep_matvec_w4(state["cfg"], state["args"], stream)
    return state["C"]


# -------------------------------------------------------------------- work


def work(case):
    op, T, k = case["op"], case["tokens"], case["top_k"]
    if op in ("route", "route_backward"):
        E, b = case["experts"], 4 if case["dtype"] == "f32" else 2
        if op == "route":
            return dict(bytes=T * E * b + T * k * 8 + (4 * E if case["bias"] else 0), flops=T * E * 4)
        dense = case["score"] == "softmax" and not case["renorm"]
        return dict(bytes=T * E * b * (2 if dense else 1) + T * k * (8 + (0 if dense else b)),
                    flops=T * E * (6 if dense else 1))
    N = case["N"]
    if op == "combine_backward":
        return dict(bytes=2 * T * N * (2 * k + 1) + 8 * T * k, flops=3 * T * k * N)
    E, K, G = case["experts"], case["K"], case["group"]
    # the experts that get a row, on average, each read once
    active = E * (1 - (1 - k / E) ** T)
    group_bytes = {"int4": 2, "int4z": 3, "e2m1": 1}[case["format"]]
    weights = N * K // 2 + N * (K // G) * group_bytes
    x_rows = T if case["act"] else T * k
    return dict(bytes=active * weights + 2 * x_rows * K + 2 * T * k * (N // 2 if case["act"] else N),
                flops=2 * T * k * N * K)


# ------------------------------------------------------------------- exact


def _exact_route(s):
    """Row by row of numpy in 64 bits: the chosen come from a sort of (masked, -value)."""
    c = s["case"]
    T, E, k, n = c["tokens"], c["experts"], c["top_k"], c["groups"]
    l = s["logits"].double().cpu().numpy()
    masked = np.isneginf(l)
    finite = np.where(masked, 0.0, l)
    with np.errstate(over="ignore"):
        if c["score"] == "sigmoid":
            score = u = np.where(masked, 0.0, 0.5 * (1 + np.tanh(finite / 2)))
        else:
            u = np.where(masked, 0.0, np.exp(finite - np.where(masked, -np.inf, l).max(1, keepdims=True)))
            score = u / u.sum(1, keepdims=True)
    v = l if s["bias"] is None else score + s["bias"].double().cpu().numpy()
    v = np.where(masked, -np.inf, v)
    if n > 1:
        base = v if s["bias"] is not None or c["group_top"] == 1 else np.where(masked, -np.inf, u)
        part = -np.sort(-base.reshape(T, n, -1), axis=-1)[..., :c["group_top"]]
        worth = part[..., 0] + np.where(np.isneginf(part[..., 1:]), 0, part[..., 1:]).sum(-1)
        kept = np.zeros((T, n), bool)
        np.put_along_axis(kept, np.argsort(-worth, 1, kind="stable")[:, :c["topk_groups"]], True, 1)
        out = ~np.repeat(kept, E // n, 1)
        # experts of the other groups come after everything, the masked ones included
        finite_v = np.where(np.isneginf(v), np.finfo(np.float64).min, v)
        v = np.where(out, -np.inf, finite_v)
    ids = np.argsort(-v, 1, kind="stable")[:, :k]
    a = np.take_along_axis(score, ids, 1)
    if c["renorm"]:
        t = a.sum(1, keepdims=True)
        a = np.divide(a, t, out=np.zeros_like(a), where=t > 0)
    return None, torch.from_numpy(a * c["scale"])


def _exact_route_backward(s):
    """The gradient of the gates' formula by automatic differentiation in 64 bits."""
    c, ids = s["case"], s["ids"].long()
    l = s["logits"].double()
    masked = l == -math.inf
    # a masked expert has the score e^-700: nothing next to the others, yet with a slope
    l = l.masked_fill(masked, -700.0).requires_grad_(True)
    if c["score"] == "softmax":
        sel = torch.log_softmax(l, -1).gather(1, ids)
        gates = torch.softmax(sel, -1) if c["renorm"] else sel.exp()
    else:
        gates = torch.sigmoid(l.gather(1, ids))
        if c["renorm"]:
            gates = gates / gates.sum(-1, keepdim=True)
    (gates * c["scale"]).backward(s["dgates"].double())
    nothing_left = masked.gather(1, ids).all(1, keepdim=True)
    return l.grad.masked_fill(masked | nothing_left & bool(c["renorm"]), 0.0)


def _exact_w4(s):
    c = s["case"]
    k, K, N, G = c["top_k"], c["K"], c["N"], c["group"]
    dev = s["W"].device
    low = torch.tensor(_E2M1 if c["format"] == "e2m1" else range(16), dtype=torch.float64, device=dev)
    x = s["x"].double()
    if c["act"]:
        x = x[torch.div(s["gather_idx"].long(), k, rounding_mode="floor")]
    off = s["offsets"].tolist()
    y = torch.empty(off[-1], N, dtype=torch.float64, device=dev)
    for e in range(c["experts"]):
        if off[e] == off[e + 1]:
            continue
        w = torch.empty(N, K, dtype=torch.float64, device=dev)
        w[:, 0::2] = low[(s["W"][e] % 16).long()]
        w[:, 1::2] = low[torch.div(s["W"][e], 16, rounding_mode="floor").long()]
        if c["format"] == "e2m1":
            scale = torch.pow(2.0, s["scales"][e].double() - 127)
        else:
            scale = s["scales"][e].double()
            z = s["zeros"][e].double() if s["zeros"] is not None else torch.full_like(scale, 8)
            w -= z.repeat_interleave(G, 1)
        w *= scale.repeat_interleave(G, 1)
        y[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w.T
    if c["act"]:
        y = torch.nn.functional.silu(y[:, :N // 2]) * y[:, N // 2:]
    return y


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "route_backward":
        return _exact_route_backward(s)
    if case["op"] == "combine_backward":
        dout = s["dout"].double()
        dgates = torch.einsum("tkn,tn->tk", s["rows"].double(), dout)
        return dgates, s["gates"].double()[..., None] * dout[:, None, :]
    return _exact_w4(s)


if __name__ == "__main__":
    rng = random.Random(0)
    for c in listed() + [draw(rng) for _ in range(6)]:
        print(c, work(c))
