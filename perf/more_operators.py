"""Cases of the norm in front of a layer, its gradient, the 8-bit activation and the layer of a
few tokens: ep_add_rmsnorm, ep_add_rmsnorm_backward, ep_swiglu_e4m3 and ep_layer_few, each in
a plain form (elementary torch operations in 32 bits, rounded once) and as a user calls it
(``own``).

Conventions of the framework: T tokens of H = ``hidden`` values, E local experts of intermediate
size I = ``inter``, top_k experts a token; rows in 8 bits are e4m3 codes (float8_e4m3fn) with
an fp32 scale for each 128 columns, weights in 8 bits have one for each 128 x 128 block.
"""

import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_TINY = 2.0 ** -126  # smallest scale


def listed():
    return [
        # one decoded token in front of a layer: pure latency
        dict(name="norm one token", op="norm", tokens=1, hidden=7168, residual="bf16",
             weight="bf16", out="bf16"),
        # ragged sizes, a residual stream in 32 bits, no piece of a row aligned
        dict(name="norm ragged 333x1111", op="norm", tokens=333, hidden=1111, residual="f32",
             weight="f32", out="both"),
        # one rank's prefill of 8192 tokens, rows for the 8-bit products: the largest call
        dict(name="norm 8192 to 8 bits", op="norm", tokens=8192, hidden=7168, residual="bf16",
             weight="bf16", out="e4m3"),
        # the decode batch's rows: a small fine-tuning step
        dict(name="norm backward 128", op="norm_backward", tokens=128, hidden=7168,
             residual="bf16", weight="bf16", through=False),
        # one rank's training batch, with the gradient that comes along the residual
        dict(name="norm backward 8192", op="norm_backward", tokens=8192, hidden=7168,
             residual="bf16", weight="bf16", through=True),
        # expert rows of a small decode batch between the two 8-bit products
        dict(name="swiglu 8 bits 64 rows", op="swiglu", rows=64, inter=2048),
        # expert rows of one rank's prefill: 8192 tokens, 8 of them a token
        dict(name="swiglu 8 bits 65536 rows", op="swiglu", rows=65536, inter=2048),
        # a layer of the smallest sizes: launches and latency
        dict(name="few tiny", op="few", tokens=1, experts=8, ranks=1, top_k=2, hidden=128,
             inter=256, dtype="bf16"),
        # one decoded token through 2 of 8 large experts
        dict(name="few one token 2 of 8", op="few", tokens=1, experts=8, ranks=1, top_k=2,
             hidden=4096, inter=14336, dtype="bf16"),
        # ragged sizes, half of the experts on another rank
        dict(name="few ragged 5 tokens", op="few", tokens=5, experts=12, ranks=2, top_k=3,
             hidden=1496, inter=1000, dtype="bf16"),
        # sequences decoded together on 8-bit weights
        dict(name="few 16 tokens 8 bits", op="few", tokens=16, experts=32, ranks=1, top_k=8,
             hidden=7168, inter=2048, dtype="e4m3"),
        # the largest batch of the few: every expert has rows
        dict(name="few 64 tokens 8 of 16", op="few", tokens=64, experts=16, ranks=1, top_k=8,
             hidden=4096, inter=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A row's length: mostly whole pieces of 8, sometimes any."""
    return _log(rng, 64, 7168) if rng.random() < 0.3 else 8 * _log(rng, 8, 896)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "swiglu", "few", "few", "few"])
    if op == "norm":
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=_width(rng),
                    residual=rng.choice(["none", "bf16", "f32"]),
                    weight=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "e4m3", "both"]))
    if op == "norm_backward":
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=_width(rng),
                    residual=rng.choice(["bf16", "f32"]), weight=rng.choice(["bf16", "f32"]),
                    through=rng.random() < 0.6)
    if op == "swiglu":
        return dict(op=op, rows=_log(rng, 1, 65536), inter=8 * _log(rng, 8, 256))
    e4m3 = rng.random() < 0.5
    experts = rng.choice([1, 4, 8, 12, 16, 32, 64])
    ranks = rng.choice([1, 1, 2])
    step = 128 if e4m3 else 8
    hidden = step * max(1, _log(rng, 128, 7168) // step)
    most = 16 * 4096 * 2048 * (2 if e4m3 else 1) // (experts * hidden)  # the largest listed weights
    inter = step * max(1, min(_log(rng, 128, 14336), most) // step)
    return dict(op=op, tokens=_log(rng, 1, 64), experts=experts, ranks=ranks,
                top_k=rng.randint(1, min(8, experts * ranks)), hidden=hidden, inter=inter,
                dtype="e4m3" if e4m3 else "bf16")


# ------------------------------------------------------------------ inputs


def _hidden_states(shape, g, dev):
    """Rows of about unit size, a few channels of which carry larger values."""
    x = torch.randn(shape, generator=g, device=dev)
    n = shape[-1]
    x[..., torch.randint(0, n, (max(1, n // 256),), generator=g, device=dev)] *= 8
    return x


def _rows_8bit(x):
    """e4m3 codes of rows and the scales of each 128 columns."""
    T, n = x.shape
    b = x.view(T, n // 128, 128)
    s = (b.abs().amax(-1) / 448).clamp(min=_TINY)
    return (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(T, n), s


def _weights_8bit(shape, size, g, dev):
    """[E][N][K] e4m3 weights of N(0, size^2) values and the scales of 128 x 128 blocks."""
    E, N, K = shape
    q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    s = torch.empty(E, N // 128, K // 128, device=dev)
    for e in range(E):
        w = (torch.randn(N // 128, 128, K // 128, 128, generator=g, device=dev) * size)
        s[e] = w.abs().amax((1, 3)) / 448
        q[e] = (w / s[e][:, None, :, None]).clamp(-448, 448).view(N, K).to(torch.float8_e4m3fn)
    return q, s


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_backward"):
        T, H = case["tokens"], case["hidden"]
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device=dev)).to(_DTYPES[case["weight"]])
        stream = _DTYPES["bf16" if case["residual"] == "none" else case["residual"]]
        if op == "norm":
            s["x"] = _hidden_states((T, H), g, dev).bfloat16()
            s["residual"] = None
            if case["residual"] != "none":
                s["residual"] = (3 * _hidden_states((T, H), g, dev)).to(stream)
                s["sum"] = torch.empty(T, H, dtype=stream, device=dev)
            if case["out"] != "e4m3":
                s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
            if case["out"] != "bf16":
                s["q"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=dev)
                s["q_scales"] = torch.empty(T, (H + 127) // 128, device=dev)
        else:
            s["h"] = (3 * _hidden_states((T, H), g, dev)).to(stream)
            s["dy"] = (0.1 * torch.randn(T, H, generator=g, device=dev)).bfloat16()
            s["dsum"] = (0.1 * torch.randn(T, H, generator=g, device=dev)).to(stream) \
                if case["through"] else None
            s["dh"] = torch.empty_like(s["h"])
            s["dweight"] = torch.empty(H, device=dev)
    elif op == "swiglu":
        M, I = case["rows"], case["inter"]
        s["G"] = torch.randn(M, 2 * I, generator=g, device=dev).bfloat16()
        s["offsets"] = torch.tensor([0, M], dtype=torch.int32, device=dev)
        s["q"] = torch.empty(M, I, dtype=torch.float8_e4m3fn, device=dev)
        s["q_scales"] = torch.empty(M, (I + 127) // 128, device=dev)
    else:
        T, E, R, k = case["tokens"], case["experts"], case["ranks"], case["top_k"]
        H, I = case["hidden"], case["inter"]
        x = _hidden_states((T, H), g, dev)
        score = torch.rand(T, R * E, generator=g, device=dev)
        s["ids"] = score.argsort(dim=1)[:, :k].to(torch.int32).contiguous()
        s["gates"] = torch.softmax(torch.randn(T, k, generator=g, device=dev), -1)
        if case["dtype"] == "e4m3":
            s["x"], s["x_scales"] = _rows_8bit(x)
            s["W1"], s["w1_scales"] = _weights_8bit((E, 2 * I, H), H ** -0.5, g, dev)
            s["W2"], s["w2_scales"] = _weights_8bit((E, H, I), I ** -0.5, g, dev)
        else:
            s["x"] = x.bfloat16()
            s["W1"] = torch.randn(E, 2 * I, H, generator=g, device=dev, dtype=torch.bfloat16) * H ** -0.5
            s["W2"] = torch.randn(E, H, I, generator=g, device=dev, dtype=torch.bfloat16) * I ** -0.5
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:
        _handle(s)
    return s


_EPS = 1e-6


def _handle(s):
    """The argument blocks a program keeps for its calls: pointers and sizes only."""
    import moe_expert_gemm_gb300 as ep

    case, op = s["case"], s["case"]["op"]
    T = case.get("tokens", 1)
    k = case.get("top_k", 1)
    K = case.get("inter", 64) if op == "few" else 64
    N = case.get("hidden", 64) if op == "few" else 64
    cfg = ep.ep_config(n_ranks=case.get("ranks", 1), my_rank=case.get("ranks", 1) - 1,
                       n_local_experts=case.get("experts", 1), top_k=k, num_tokens=T,
                       max_tokens_per_rank=T, K=K, N=N, msg_bytes=2 * N,
                       dtype=ep.EP_FP8_1D2D if case.get("dtype") == "e4m3" else ep.EP_BF16,
                       send_warps=-1, signal_mode=0)
    rows = {torch.float32: ep.EP_ROWS_F32, torch.bfloat16: ep.EP_ROWS_BF16}
    p = ep.ptr
    if op == "norm":
        a = ep.ep_add_rmsnorm_args(x=p(s["x"]), residual=p(s["residual"]), weight=p(s["weight"]),
                                   weight_dtype=rows[s["weight"].dtype], hidden=case["hidden"],
                                   eps=_EPS, y=p(s.get("y")), q=p(s.get("q")),
                                   q_scales=p(s.get("q_scales")))
        if s["residual"] is not None:
            a.sum, a.residual_dtype = p(s["sum"]), rows[s["residual"].dtype]
    elif op == "norm_backward":
        size = ep.ep_add_rmsnorm_backward_sizes(cfg, case["hidden"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["h"].device)
        a = ep.ep_add_rmsnorm_backward_args(h=p(s["h"]), h_dtype=rows[s["h"].dtype], dy=p(s["dy"]),
                                            dsum=p(s["dsum"]), weight=p(s["weight"]),
                                            weight_dtype=rows[s["weight"].dtype],
                                            hidden=case["hidden"], eps=_EPS, dh=p(s["dh"]),
                                            dweight=p(s["dweight"]), workspace=p(s["workspace"]),
                                            workspace_bytes=size)
    elif op == "swiglu":
        a = ep.ep_swiglu_e4m3_args(G=p(s["G"]), q=p(s["q"]), q_scales=p(s["q_scales"]),
                                   expert_offsets=p(s["offsets"]), max_rows=case["rows"],
                                   inter=case["inter"])
    else:
        size = ep.ep_layer_few_sizes(cfg)
        # zero before the first call; every call leaves it ready for the next
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=s["x"].device)
        a = ep.ep_layer_few_args(x=p(s["x"]), x_scales=p(s.get("x_scales")), topk_ids=p(s["ids"]),
                                 gates=p(s["gates"]), W1=p(s["W1"]),
                                 w1_scales=p(s.get("w1_scales")), W2=p(s["W2"]),
                                 w2_scales=p(s.get("w2_scales")), out=p(s["out"]),
                                 workspace=p(s["workspace"]), workspace_bytes=size,
                                 status=p(s["status"]))
    s["ep"], s["cfg"], s["args"] = ep, cfg, a


# --------------------------------------------------------------- plain form


def _plain_8bit(y):
    """Codes and scales of rows whose length need not be whole groups of 128."""
    T, n = y.shape
    groups = (n + 127) // 128
    b = torch.zeros(T, groups * 128, device=y.device)
    b[:, :n] = y
    b = b.view(T, groups, 128)
    s = (b.abs().amax(-1) / 448).clamp(min=_TINY)
    q = (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(T, -1)
    return q[:, :n].contiguous(), s


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        out["sum"] = h.to(s["residual"].dtype)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + _EPS)
    y = h * r * s["weight"].float()
    if s["case"]["out"] != "e4m3":
        out["y"] = y.bfloat16()
    if s["case"]["out"] != "bf16":
        out["q"], out["q_scales"] = _plain_8bit(y)
    return out


def _plain_norm_backward(s):
    h, dy = s["h"].float(), s["dy"].float()
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + _EPS)
    g = dy * s["weight"].float()
    dh = r * (g - h * (r * r * (g * h).mean(-1, keepdim=True)))
    if s["dsum"] is not None:
        dh = dh + s["dsum"].float()
    # (a sum over up to thousands of tokens)
    dweight = (dy * h * r).double().sum(0).float()
    return {"dh": dh.to(s["h"].dtype), "dweight": dweight}


def _silu_times(gate, up):
    return gate / (1 + torch.exp(-gate)) * up


def _plain_swiglu(s):
    I = s["case"]["inter"]
    q, scales = _plain_8bit(_silu_times(s["G"][:, :I].float(), s["G"][:, I:].float()))
    return {"q": q, "q_scales": scales}


def _wide_rows(q, scales):
    return q.float() if scales is None else \
        (q.float().view(q.shape[0], -1, 128) * scales[..., None]).view(q.shape)


def _wide_weights(q, scales):
    if scales is None:
        return q.float()
    E, N, K = q.shape
    return (q.float().view(E, N // 128, 128, K // 128, 128) * scales[:, :, None, :, None]).view(E, N, K)


def _plain_few(s):
    c = s["case"]
    T, E, k, I = c["tokens"], c["experts"], c["top_k"], c["inter"]
    x = _wide_rows(s["x"], s.get("x_scales"))
    # the rank's own experts are the last ones
    local = s["ids"].long().view(-1) - (c["ranks"] - 1) * E
    there = local >= 0
    at = local.clamp(min=0)
    w1_scales, w2_scales = s.get("w1_scales"), s.get("w2_scales")
    pick = (lambda w: None if w is None else w[at]) if T * k <= E else (lambda w: w)
    w1 = _wide_weights(pick(s["W1"]), pick(w1_scales))
    w2 = _wide_weights(pick(s["W2"]), pick(w2_scales))
    token = torch.arange(T * k, device=x.device) // k
    if T * k <= E:  # every row by weights of its own
        gu = torch.bmm(x[token][:, None, :], w1.transpose(1, 2))[:, 0]
    else:  # every expert's rows in a block of T rows (it has at most one of each token)
        gu = torch.matmul(x, w1.transpose(1, 2)).view(E * T, 2 * I)[at * T + token]
    a = _silu_times(gu[:, :I], gu[:, I:])
    # the activation meets the second product in the operands' type
    a = a.bfloat16().float() if c["dtype"] == "bf16" else _wide_rows(*_plain_8bit(a))
    if T * k <= E:
        y = torch.bmm(a[:, None, :], w2.transpose(1, 2))[:, 0]
    else:
        rows = torch.zeros(E * T, I, device=x.device)
        rows[(at * T + token)[there]] = a[there]
        y = torch.bmm(rows.view(E, T, I), w2.transpose(1, 2)).view(E * T, -1)[at * T + token]
    y = torch.where(there[:, None], y, torch.zeros_like(y)).view(T, k, -1)
    return {"out": (s["gates"][..., None] * y).sum(1).bfloat16()}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "swiglu": _plain_swiglu,
          "few": _plain_few}


def run(state):
    op = state["case"]["op"]
    if not own:
        return _PLAIN[op](state)
    ep, stream = state["ep"], torch.cuda.current_stream()
    if op == "norm":
        ep.ep_add_rmsnorm(state["cfg"], state["args"], stream)
        return {n: state[n] for n in ("sum", "y", "q", "q_scales") if n in state}
    if op == "norm_backward":
        ep.ep_add_rmsnorm_backward(state["cfg"], state["args"], stream)
        return {"dh": state["dh"], "dweight": state["dweight"]}
    if op == "swiglu":
        ep.ep_swiglu_e4m3(state["cfg"], state["args"], stream)
        return {"q": state["q"], "q_scales": state["q_scales"]}
    ep.ep_layer_few(state["cfg"], state["args"], stream)
    return {"out": state["out"]}


# -------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, H = case["tokens"], case["hidden"]
        stream = {"none": 0, "bf16": 2, "f32": 4}[case["residual"]]
        weight = H * (2 if case["weight"] == "bf16" else 4)
        if op == "norm":
            out = {"bf16": 2, "e4m3": 1, "both": 3}[case["out"]]
            scales = 0 if case["out"] == "bf16" else 4 * T * ((H + 127) // 128)
            return dict(bytes=T * H * (2 + 2 * stream + out) + scales + weight, flops=6 * T * H)
        return dict(bytes=T * H * (2 + stream * (3 if case["through"] else 2)) + weight + 4 * H,
                    flops=12 * T * H)
    if op == "swiglu":
        M, I = case["rows"], case["inter"]
        return dict(bytes=M * (5 * I + 4 * ((I + 127) // 128)), flops=8 * M * I)
    T, E, R, k = case["tokens"], case["experts"], case["ranks"], case["top_k"]
    H, I, b = case["hidden"], case["inter"], 2 if case["dtype"] == "bf16" else 1
    # the local experts that get a row, on average, each read once
    active = E * (1 - (1 - k / (E * R)) ** T)
    return dict(bytes=active * 3 * H * I * b + T * H * (b + 2) + 8 * T * k,
                flops=6 * T * k / R * H * I)


# ------------------------------------------------------------------- exact


def _exact_8bit(y):
    """The numbers that the codes of rows round, and the scales."""
    T, n = y.shape
    pad = torch.nn.functional.pad(y, (0, -n % 128)).unflatten(1, (-1, 128))
    s = pad.abs().amax(2).div(448).clamp(min=_TINY)
    return pad.div(s.unsqueeze(2)).flatten(1)[:, :n], s


def _to_e4m3(v):
    """Nearest e4m3 numbers, ties to even, by the format's definition."""
    a = v.abs().clamp(max=448)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448)


def _exact_few(s):
    """Expert by expert: its tokens through its two matrices."""
    c = s["case"]
    T, E, I, H = c["tokens"], c["experts"], c["inter"], c["hidden"]

    def weights(name, e):
        w = s[name][e].double()
        if c["dtype"] == "e4m3":
            sc = s[name.lower() + "_scales"][e].double()
            w = w * sc.repeat_interleave(128, 0).repeat_interleave(128, 1)
        return w

    x = s["x"].double()
    if c["dtype"] == "e4m3":
        x = x * s["x_scales"].double().repeat_interleave(128, 1)
    ids, out = s["ids"].cpu(), torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(ids == e + (c["ranks"] - 1) * E, as_tuple=True)
        if not len(t):
            continue
        t, j = t.to(x.device), j.to(x.device)
        gu = x[t] @ weights("W1", e).T
        a = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        if c["dtype"] == "e4m3":
            v, sc = _exact_8bit(a)
            a = _to_e4m3(v) * sc.repeat_interleave(128, 1)
        else:
            a = a.bfloat16().double()
        out.index_add_(0, t, s["gates"][t, j].double()[:, None] * (a @ weights("W2", e).T))
    return {"out": out}


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    op = case["op"]
    if op == "few":
        # (64-bit products of the largest draws would take long)
        active = min(case["experts"], case["tokens"] * case["top_k"])
        if active * case["hidden"] * case["inter"] > 2 ** 31:
            return None
        return _exact_few(s)
    if op == "swiglu":
        gate, up = s["G"].double().chunk(2, 1)
        v, scales = _exact_8bit(torch.sigmoid(gate) * gate * up)
        return {"q": v, "q_scales": scales}
    w = s["weight"].double()
    if op == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["sum"] = h
        y = h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + _EPS) * w
        if case["out"] != "e4m3":
            out["y"] = y
        if case["out"] != "bf16":
            out["q"], out["q_scales"] = _exact_8bit(y)
        return out
    # the gradient of the norm's formula by automatic differentiation
    h, w = s["h"].double().requires_grad_(True), w.requires_grad_(True)
    (h / torch.sqrt(h.pow(2).mean(1, keepdim=True) + _EPS) * w).backward(s["dy"].double())
    dh = h.grad if s["dsum"] is None else h.grad + s["dsum"].double()
    return {"dh": dh, "dweight": w.grad}


if __name__ == "__main__":
    rng = random.Random(0)
    for c in listed() + [draw(rng) for _ in range(6)]:
        print(c, work(c))
