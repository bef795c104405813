"""Device state of a set of logical EP ranks on one GPU, driven through the C ABI.

PyTorch only allocates device memory and provides streams; every step runs in
``libmoe_ep.so``. On one GPU the receive buffers of the other logical ranks
are separate allocations in the same HBM that stand in for peer memory, so a
producer call for rank r writes into every rank's buffer exactly as it would
over direct peer stores.
"""

from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import (EP_ACT_NONE, EP_ACT_SWIGLU, EP_BF16, EP_FP8_1D2D, EP_LOGITS_BF16, EP_LOGITS_F32,
               EP_SCORE_SOFTMAX, EP_W4_E2M1, EP_W4_INT, ep_combine_args, ep_combine_backward,
               ep_combine_backward_args, ep_combine_reduce, ep_config, ep_dispatch_args,
               ep_dispatch_gather, ep_matvec_w4, ep_matvec_w4_sizes, ep_plan, ep_plan_out,
               ep_plan_sizes, ep_route, ep_route_args, ep_route_backward, ep_route_backward_args,
               ep_scatter_args, ep_scatter_send, ep_send_args, ep_swiglu, ep_swiglu_args,
               ep_w4_args, grouped_gemm_combine_send, ptr)
from .w4 import W4Weights

SENTINEL_BYTE = 0xFF  # received bf16 0xFFFF is a NaN: an unwritten slot cannot pass
STATUS_PLAN, STATUS_SEND, STATUS_COMBINE, STATUS_ROUTE, STATUS_W4 = 0, 1, 2, 3, 4


def _check_flat(name: str, t: torch.Tensor, count: int, dtype: torch.dtype, device: torch.device):
    """The kernels go by address and size: a tensor of another type, size or device, or with
    gaps or repeats in memory, would be read as something else or past its end."""
    if t.dtype != dtype or t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{name}: {count} contiguous elements of {dtype} expected, got "
                         f"{tuple(t.shape)} of {t.dtype} with strides {t.stride()}")
    if t.device.type != device.type or device.index not in (None, t.device.index):
        raise ValueError(f"{name}: on {t.device}, expected on {device}")


def _check_rows(name: str, t: torch.Tensor, rows: int, cols: int, dtypes, device: torch.device) -> int:
    """Of a [rows][cols] tensor whose rows may lie any stride apart: that stride, as the calls
    take it (0: back to back)."""
    if tuple(t.shape) != (rows, cols) or t.dtype not in dtypes:
        raise ValueError(f"{name}: [{rows}][{cols}] of {' or '.join(map(str, dtypes))} expected, "
                         f"got {tuple(t.shape)} of {t.dtype}")
    if t.device.type != device.type or device.index not in (None, t.device.index):
        raise ValueError(f"{name}: on {t.device}, expected on {device}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row lie {t.stride(1)} apart")
    if rows <= 1:
        return 0  # (a single row's stride says nothing)
    if t.stride(0) < cols:
        raise ValueError(f"{name}: rows of {cols} elements lie {t.stride(0)} apart")
    return t.stride(0)


class EpSystem:
    def __init__(self, n_ranks: int, n_local_experts: int, top_k: int, tokens: int, K: int,
                 N: int, dtype: str = "bf16", device="cuda", max_tokens: int | None = None,
                 timeout_ns: int = 0, send_warps: int = -1, signal_mode: int = 0):
        self.R, self.El, self.k, self.T, self.K, self.N = (n_ranks, n_local_experts, top_k,
                                                           tokens, K, N)
        self.dtype = dtype
        self.dt_code = {"bf16": EP_BF16, "fp8_1d2d": EP_FP8_1D2D}[dtype]
        self.device = torch.device(device)
        self.max_tokens = tokens if max_tokens is None else max_tokens
        self.msg_bytes = 2 * N
        self.timeout_ns = timeout_ns
        self.send_warps = send_warps
        self.signal_mode = signal_mode  # EP_SIGNAL_RANK_FLAG or EP_SIGNAL_PER_EXPERT
        dev = self.device
        R, El = self.R, self.El
        self.recv = [torch.full((self.max_tokens * top_k * self.msg_bytes,), SENTINEL_BYTE,
                                dtype=torch.uint8, device=dev) for _ in range(R)]
        self.counts = [torch.full((El * R + R,), -1, dtype=torch.int64, device=dev)
                       for _ in range(R)]
        self.atomic_counter = [torch.zeros(El, dtype=torch.int32, device=dev) for _ in range(R)]
        self.rank_counter = [torch.zeros(R, dtype=torch.int32, device=dev) for _ in range(R)]
        self.block_counter = [torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(R)]
        self.status = torch.zeros(8, dtype=torch.int32, device=dev)
        self.topk = None
        self._route_ids = torch.zeros((R, tokens, top_k), dtype=torch.int32, device=dev)
        self.plans: list[dict | None] = [None] * R
        self.ops: list[dict | None] = [None] * R
        self.gates: list[torch.Tensor | None] = [None] * R
        self.out: list[torch.Tensor | None] = [None] * R
        self.routes: list[dict | None] = [None] * R
        self.layer_w4: list[dict | None] = [None] * R

    # ------------------------------------------------------------- set-up
    def cfg(self, rank: int) -> ep_config:
        return ep_config(self.R, rank, self.El, self.k, self.T, self.max_tokens, self.K, self.N,
                         self.msg_bytes, self.dt_code, self.send_warps, self.signal_mode)

    def _on(self, stream):
        """What a call makes for itself is allocated and filled inside this context: on the
        stream its kernel goes to, ahead of it. (On torch's current stream the fill could land
        after the kernel, and the caller can order nothing inside one call.)"""
        if self.device.type != "cuda":
            return contextlib.nullcontext()
        if stream is None or stream == 0:
            stream = torch.cuda.default_stream(self.device)
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, self.device)
        return torch.cuda.stream(stream)

    def reset_buffers(self):
        for b in self.recv:
            b.fill_(SENTINEL_BYTE)
        for c in self.counts:
            c.fill_(-1)

    def set_routing(self, topk_ids):
        t = torch.as_tensor(np.ascontiguousarray(topk_ids, dtype=np.int32))
        assert tuple(t.shape) == (self.R, self.T, self.k)
        self.topk = t.to(self.device)

    def plan(self, rank: int, stream=None, max_rows: int | None = None) -> dict:
        cap = ep_plan_sizes(self.cfg(rank)) if max_rows is None else max_rows
        dev, El, R = self.device, self.El, self.R
        with self._on(stream):
            p = dict(expert_offsets=torch.zeros(El + 1, dtype=torch.int32, device=dev),
                     src_info=torch.zeros((max(cap, 1), 2), dtype=torch.int32, device=dev),
                     seg_offsets=torch.zeros((El, R + 1), dtype=torch.int32, device=dev),
                     send_counts=torch.zeros((El, R), dtype=torch.int32, device=dev),
                     gather_idx=torch.zeros(max(cap, 1), dtype=torch.int32, device=dev),
                     m_total=torch.zeros(1, dtype=torch.int32, device=dev), capacity=cap)
        out = ep_plan_out(ptr(p["expert_offsets"]), ptr(p["src_info"]), ptr(p["seg_offsets"]),
                          ptr(p["send_counts"]), ptr(p["gather_idx"]), ptr(p["m_total"]),
                          self.status.data_ptr() + 4 * STATUS_PLAN, cap)
        ep_plan(self.cfg(rank), self.topk, out, stream)
        self.plans[rank] = p
        return p

    def set_operands(self, rank: int, A: np.ndarray, W: np.ndarray, a_scales=None,
                     w_scales=None, pad_rows: int = 0):
        """Upload a rank's operands (bf16 as uint16 bit patterns, e4m3 as uint8).
        ``pad_rows`` extra rows are appended to A (they are read by tiles that run
        past the last row and never sent)."""
        dev = self.device
        rows = max(A.shape[0] + pad_rows, 1)
        if self.dtype == "bf16":
            a = torch.zeros((rows, self.K), dtype=torch.int16)
            a[:A.shape[0]] = torch.from_numpy(np.ascontiguousarray(A).view(np.int16))
            w = torch.from_numpy(np.ascontiguousarray(W).view(np.int16))
            ops = dict(A=a.view(torch.bfloat16).to(dev), W=w.view(torch.bfloat16).to(dev))
        else:
            a = torch.zeros((rows, self.K), dtype=torch.uint8)
            a[:A.shape[0]] = torch.from_numpy(np.ascontiguousarray(A))
            sa = torch.zeros((rows, self.K // 128), dtype=torch.float32)
            sa[:A.shape[0]] = torch.from_numpy(np.ascontiguousarray(a_scales, dtype=np.float32))
            ops = dict(A=a.to(dev), W=torch.from_numpy(np.ascontiguousarray(W)).to(dev),
                       a_scales=sa.to(dev),
                       w_scales=torch.from_numpy(np.ascontiguousarray(w_scales,
                                                                      dtype=np.float32)).to(dev))
        self.ops[rank] = ops
        return ops

    def set_gates(self, rank: int, gates: np.ndarray):
        self.gates[rank] = torch.from_numpy(np.ascontiguousarray(gates, dtype=np.float32)).to(
            self.device)
        self.out[rank] = torch.zeros((self.T, self.N), dtype=torch.bfloat16, device=self.device)

    # ---------------------------------------------------------------- calls
    def send_args(self, rank: int, epoch: int, p3_control: int = 0, C=None) -> ep_send_args:
        p, o = self.plans[rank], self.ops[rank]
        a = ep_send_args()
        a.A = ptr(o["A"])
        a.a_scales = ptr(o.get("a_scales"))
        a.W = ptr(o["W"])
        a.w_scales = ptr(o.get("w_scales"))
        a.expert_offsets = ptr(p["expert_offsets"])
        a.src_info = ptr(p["src_info"])
        a.seg_offsets = ptr(p["seg_offsets"])
        a.send_counts = ptr(p["send_counts"])
        a.max_rows = min(int(o["A"].shape[0]), int(p["src_info"].shape[0]))
        for d in range(self.R):
            a.recv_buf_ptrs[d] = ptr(self.recv[d])
            a.recv_count_ptrs[d] = ptr(self.counts[d])
        a.atomic_counter = ptr(self.atomic_counter[rank])
        a.rank_completion_counter = ptr(self.rank_counter[rank])
        a.epoch = epoch
        a.p3_control = p3_control
        a.C = ptr(C)
        a.status = self.status.data_ptr() + 4 * STATUS_SEND
        a.trace = None
        a.timeout_ns = self.timeout_ns
        return a

    def send(self, rank: int, epoch: int, stream=None, p3_control: int = 0, C=None,
             overlap: bool = False):
        """``overlap``: may start while the kernel before it on the stream is still
        finishing (programmatic dependent launch; it reads nothing before that kernel
        has completed)."""
        a = self.send_args(rank, epoch, p3_control, C)
        a.overlap_previous = 1 if overlap else 0
        grouped_gemm_combine_send(self.cfg(rank), a, stream)

    def local_C(self, rank: int):
        """A [max_rows][N] bf16 buffer for the unfused path's local GEMM output."""
        return torch.empty((self.ops[rank]["A"].shape[0], self.N), dtype=torch.bfloat16,
                           device=self.device)

    def send_unfused(self, rank: int, epoch: int, C, stream=None):
        """The unfused comparator: the grouped GEMM with the sink disabled stores its
        rows to the local C, then ep_scatter_send moves them and signals."""
        grouped_gemm_combine_send(self.cfg(rank), self.send_args(rank, epoch, -1, C), stream)
        ep_scatter_send(self.cfg(rank), self.scatter_args(rank, epoch, C), stream)

    def scatter_args(self, rank: int, epoch: int, C) -> ep_scatter_args:
        p = self.plans[rank]
        a = ep_scatter_args()
        a.C = ptr(C)
        a.expert_offsets = ptr(p["expert_offsets"])
        a.src_info = ptr(p["src_info"])
        a.seg_offsets = ptr(p["seg_offsets"])
        a.send_counts = ptr(p["send_counts"])
        a.max_rows = min(int(C.shape[0]), int(p["src_info"].shape[0]))
        for d in range(self.R):
            a.recv_buf_ptrs[d] = ptr(self.recv[d])
            a.recv_count_ptrs[d] = ptr(self.counts[d])
        a.block_counter = ptr(self.block_counter[rank])
        a.epoch = epoch
        a.status = self.status.data_ptr() + 4 * STATUS_SEND
        return a

    # ------------------------------------------------------------ whole layer
    def set_layer_operands(self, rank: int, X: np.ndarray, W1: np.ndarray, W2: np.ndarray):
        """Operands of a whole MoE layer around the down-projection (bf16 bit
        patterns): the rank's tokens X [T, H], its experts' up/gate weights W1
        [E_l, 2I, H] (gate rows first) and down-projection weights W2 [E_l, H, I],
        with H = N and I = K. The down-projection's A is produced on the device by
        layer_forward (dispatch, up/gate GEMM, activation)."""
        assert self.dtype == "bf16"
        dev, H, I = self.device, self.N, self.K
        x = torch.zeros((self.max_tokens, H), dtype=torch.int16)
        x[:X.shape[0]] = torch.from_numpy(np.ascontiguousarray(X).view(np.int16))
        rows = max(self.plans[rank]["capacity"], 1)
        self.layer = getattr(self, "layer", [None] * self.R)
        w1 = np.ascontiguousarray(W1).view(np.int16)
        # the same rows in 128-row gate/up blocks, for the activation in the epilogue
        El = w1.shape[0]
        w1i = w1.reshape(El, 2, I // 128, 128, H).transpose(0, 2, 1, 3, 4).reshape(El, 2 * I, H) \
            if I % 128 == 0 else None
        self.layer[rank] = dict(
            X=x.view(torch.bfloat16).to(dev),
            W1=torch.from_numpy(w1).view(torch.bfloat16).to(dev),
            W1i=None if w1i is None else torch.from_numpy(np.ascontiguousarray(w1i)).view(
                torch.bfloat16).to(dev),
            A_in=torch.zeros((rows, H), dtype=torch.bfloat16, device=dev),
            G=torch.zeros((rows, 2 * I), dtype=torch.bfloat16, device=dev))
        self.ops[rank] = dict(
            A=torch.zeros((rows, I), dtype=torch.bfloat16, device=dev),
            W=torch.from_numpy(np.ascontiguousarray(W2).view(np.int16)).view(
                torch.bfloat16).to(dev))

    def cfg_up(self, rank: int) -> ep_config:
        """The up/gate projection's configuration: K = H, N = 2I."""
        return ep_config(self.R, rank, self.El, self.k, self.T, self.max_tokens, self.N,
                         2 * self.K, 4 * self.K, EP_BF16, self.send_warps, self.signal_mode)

    def layer_forward(self, rank: int, epoch: int, stream=None, p3_control: int = 0,
                      events=None, fused_act: bool = False, overlap: bool = False):
        """Dispatch, up/gate GEMM, activation, then the fused down-projection + send
        of producer ``rank`` (every ``layer[r]["X"]`` must hold rank r's tokens).
        ``fused_act``: the activation runs in the up/gate GEMM's epilogue (interleaved
        W1, no G) instead of as its own pass. ``events``: four CUDA events recorded
        after each of the first four steps. ``overlap``: the two GEMM calls launch as
        programmatic dependents of the kernel before them (their set-up overlaps its
        end); ignored when ``events`` are recorded between the steps."""
        L, p = self.layer[rank], self.plans[rank]
        mark = (lambda i: events[i].record(stream)) if events is not None else (lambda i: None)
        d = ep_dispatch_args()
        for r in range(self.R):
            d.x_ptrs[r] = ptr(self.layer[r]["X"])
        d.gather_idx = ptr(p["gather_idx"])
        d.expert_offsets = ptr(p["expert_offsets"])
        d.max_rows = int(L["A_in"].shape[0])
        d.hidden = self.N
        d.A_in = ptr(L["A_in"])
        d.status = self.status.data_ptr() + 4 * STATUS_SEND
        ep_dispatch_gather(self.cfg(rank), d, stream)
        mark(0)
        up = self.send_args(rank, epoch, -1, self.ops[rank]["A"] if fused_act else L["G"])
        up.A = ptr(L["A_in"])
        up.W = ptr(L["W1i"] if fused_act else L["W1"])
        up.max_rows = int(L["A_in"].shape[0])
        if fused_act:
            up.local_activation = EP_ACT_SWIGLU
        overlap = overlap and events is None
        up.overlap_previous = 1 if overlap else 0
        grouped_gemm_combine_send(self.cfg_up(rank), up, stream)
        mark(1)
        if not fused_act:
            a = ep_swiglu_args(ptr(L["G"]), ptr(self.ops[rank]["A"]),
                               ptr(p["expert_offsets"]), int(L["G"].shape[0]), self.K)
            ep_swiglu(self.cfg(rank), a, stream)
        mark(2)
        self.send(rank, epoch, stream, p3_control=p3_control, overlap=overlap)
        mark(3)

    # ------------------------------------------------- routing and its gradient
    def route(self, rank: int, logits: torch.Tensor, score: int = EP_SCORE_SOFTMAX, bias=None,
              n_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
              renormalize: bool = True, scale: float = 1.0, stream=None):
        """The rank's routing and gates on the device, from its router's logits [T][E]
        (fp32 or bf16, rows any stride of at least E apart) and an fp32 bias [E]: in place of
        ``set_routing`` and ``set_gates``. Every rank's routing stands before any rank's ``plan``."""
        E = self.R * self.El
        stride = _check_rows("logits", logits, self.T, E, self._LOGITS, self.device)
        if bias is not None:
            _check_flat("bias", bias, E, torch.float32, self.device)
        if self.topk is None:
            self.topk = self._route_ids  # of all ranks, whose calls may go to streams of their own
        if self.gates[rank] is None:
            with self._on(stream):
                self.gates[rank] = torch.zeros((self.T, self.k), device=self.device)
        if self.out[rank] is None:
            with self._on(stream):
                self.out[rank] = torch.zeros((self.T, self.N), dtype=torch.bfloat16,
                                             device=self.device)
        a = ep_route_args(logits=ptr(logits), logits_stride=stride,
                          logits_dtype=self._LOGITS[logits.dtype], score=score, bias=ptr(bias),
                          n_groups=n_groups, topk_groups=topk_groups, group_top=group_top,
                          renormalize=int(renormalize), scale=scale,
                          topk_ids=ptr(self.topk[rank]), gates=ptr(self.gates[rank]))
        ep_route(self.cfg(rank), a, stream)
        self.routes[rank] = dict(logits=logits, stride=stride, score=score,
                                 renormalize=int(renormalize), scale=scale)

    _LOGITS = {torch.float32: EP_LOGITS_F32, torch.bfloat16: EP_LOGITS_BF16}

    def combine_backward(self, rank: int, dout: torch.Tensor, dgates=None, drows=None,
                         stream=None):
        """Gradients of ``combine``'s sum for its output's gradient ``dout`` [T][N] bf16, of the
        gates ([T][k] fp32) and of the rows ([T][k][N] bf16, or the rank's receive buffer),
        each into a tensor that is given. All of them contiguous."""
        _check_flat("dout", dout, self.T * self.N, torch.bfloat16, self.device)
        if dgates is not None:
            _check_flat("dgates", dgates, self.T * self.k, torch.float32, self.device)
        if drows is not None and drows is not self.recv[rank]:
            _check_flat("drows", drows, self.T * self.k * self.N, torch.bfloat16, self.device)
        a = ep_combine_backward_args(recv_buf=ptr(self.recv[rank]), gates=ptr(self.gates[rank]),
                                     dout=ptr(dout), dgates=ptr(dgates), drows=ptr(drows))
        ep_combine_backward(self.cfg(rank), a, stream)

    def route_backward(self, rank: int, dgates: torch.Tensor, dlogits: torch.Tensor, stream=None):
        """Gradient of the logits of ``route``'s last call, which must still stand, from the
        gates' ([T][k] fp32, contiguous); into ``dlogits`` (their type and shape, rows any stride
        of at least E apart)."""
        r = self.routes[rank]
        _check_flat("dgates", dgates, self.T * self.k, torch.float32, self.device)
        stride = _check_rows("dlogits", dlogits, self.T, self.R * self.El, (r["logits"].dtype,),
                             self.device)
        a = ep_route_backward_args(logits=ptr(r["logits"]), logits_stride=r["stride"],
                                   logits_dtype=self._LOGITS[r["logits"].dtype],
                                   score=r["score"], renormalize=r["renormalize"],
                                   scale=r["scale"], topk_ids=ptr(self.topk[rank]),
                                   dgates=ptr(dgates), dlogits=ptr(dlogits),
                                   dlogits_stride=stride,
                                   status=self.status.data_ptr() + 4 * STATUS_ROUTE)
        ep_route_backward(self.cfg(rank), a, stream)

    # --------------------------------------------- a layer of few tokens, 4 bits
    def set_layer_w4(self, rank: int, X: torch.Tensor, W1: W4Weights, W2: W4Weights):
        """Operands of a MoE layer on 4-bit weights: the rank's tokens X
        [max_tokens][H] bf16, its experts' up/gate weights W1 ([E_l][2I] rows of H, gate rows
        first) and down-projection weights W2 ([E_l][H] rows of I), with H = N and I = K; all
        contiguous. Allocates the layer's buffers and its two workspaces, on torch's current
        stream."""
        assert self.dtype == "bf16" and tuple(X.shape) == (self.max_tokens, self.N)
        _check_flat("X", X, self.max_tokens * self.N, torch.bfloat16, self.device)
        self._check_w4("W1", W1, self.El * 2 * self.K, self.N)
        self._check_w4("W2", W2, self.El * self.N, self.K)
        dev, rows = self.device, max(ep_plan_sizes(self.cfg(rank)), 1)
        self.layer_w4[rank] = dict(
            X=X, W1=W1, W2=W2,
            A=torch.zeros((rows, self.K), dtype=torch.bfloat16, device=dev),
            C=torch.zeros((rows, self.N), dtype=torch.bfloat16, device=dev),
            workspaces=[torch.zeros(ep_matvec_w4_sizes(c), dtype=torch.uint8, device=dev)
                        for c in (self.cfg_up(rank), self.cfg(rank))])

    def _check_w4(self, name: str, w: W4Weights, rows: int, cols: int):
        if w.group_size < 1 or cols % w.group_size:
            raise ValueError(f"{name}: groups of {w.group_size} in rows of {cols}")
        if w.w_format not in (EP_W4_INT, EP_W4_E2M1):
            raise ValueError(f"{name}: w_format {w.w_format}")
        groups = rows * (cols // w.group_size)
        _check_flat(f"{name}.codes", w.codes, rows * cols // 2, torch.uint8, self.device)
        _check_flat(f"{name}.scales", w.scales, groups,
                    torch.uint8 if w.w_format == EP_W4_E2M1 else torch.bfloat16, self.device)
        if w.zeros is not None:
            _check_flat(f"{name}.zeros", w.zeros, groups, torch.uint8, self.device)

    def _w4_args(self, rank: int, w: W4Weights, C, workspace) -> ep_w4_args:
        p = self.plans[rank]
        return ep_w4_args(W=ptr(w.codes), w_scales=ptr(w.scales), w_zeros=ptr(w.zeros),
                          w_format=w.w_format, group_size=w.group_size,
                          expert_offsets=ptr(p["expert_offsets"]),
                          max_rows=min(int(C.shape[0]), int(p["gather_idx"].shape[0])), C=ptr(C),
                          workspace=ptr(workspace), workspace_bytes=workspace.numel(),
                          status=self.status.data_ptr() + 4 * STATUS_W4)

    def layer_forward_w4(self, rank: int, epoch: int, stream=None):
        """The layer's up/gate product with the activation in its epilogue (rows read where
        the plan finds them, no dispatch), the down-projection, and the send of producer
        ``rank`` (every ``layer_w4[r]["X"]`` must hold rank r's tokens)."""
        L = self.layer_w4[rank]
        up = self._w4_args(rank, L["W1"], L["A"], L["workspaces"][0])
        for r in range(self.R):
            up.x_ptrs[r] = ptr(self.layer_w4[r]["X"])
        up.gather_idx = ptr(self.plans[rank]["gather_idx"])
        up.local_activation = EP_ACT_SWIGLU
        ep_matvec_w4(self.cfg_up(rank), up, stream)
        down = self._w4_args(rank, L["W2"], L["C"], L["workspaces"][1])
        down.A = ptr(L["A"])
        down.local_activation = EP_ACT_NONE
        ep_matvec_w4(self.cfg(rank), down, stream)
        ep_scatter_send(self.cfg(rank), self.scatter_args(rank, epoch, L["C"]), stream)

    def send_traced(self, rank: int, epoch: int, records: int = 64, stream=None):
        """One send with per-tile timestamps; returns the decoded trace."""
        n_sm = torch.cuda.get_device_properties(self.device).multi_processor_count
        stride = 2 + 4 * records
        with self._on(stream):
            buf = torch.zeros(n_sm * stride, dtype=torch.int64, device=self.device)
        a = self.send_args(rank, epoch)
        a.trace = ptr(buf)
        a.trace_records = records
        grouped_gemm_combine_send(self.cfg(rank), a, stream)
        torch.cuda.synchronize()
        return decode_trace(buf.cpu().numpy().view(np.uint64), n_sm, records)

    def combine_args(self, rank: int, epoch: int, gates=None, out=None,
                     overlap: int = 0) -> ep_combine_args:
        g = self.gates[rank] if gates is None else gates
        o = self.out[rank] if out is None else out
        return ep_combine_args(ptr(self.recv[rank]), ptr(self.counts[rank]), ptr(g), ptr(o),
                               epoch, self.timeout_ns,
                               self.status.data_ptr() + 4 * STATUS_COMBINE,
                               ptr(self.topk[rank]) if self.topk is not None else 0,
                               int(overlap))

    def combine(self, rank: int, epoch: int, stream=None, gates=None, out=None,
                overlap: int = 0):
        """``overlap``: EP_OVERLAP_* (True is EP_OVERLAP_ANY): may start while the kernel
        before it on the stream is still finishing (programmatic dependent launch);
        EP_OVERLAP_INPUTS_READY when that kernel writes none of the gates, routing or
        output (e.g. it is the fused send)."""
        ep_combine_reduce(self.cfg(rank), self.combine_args(rank, epoch, gates, out, overlap),
                          stream)

    def publish_peer_flags(self, rank: int, epoch: int):
        """Stand-in for the other ranks finishing on their own GPUs: write the flag
        words of every source rank except ``rank`` in ``rank``'s count buffer."""
        base = self.El * self.R
        idx = [base + q for q in range(self.R) if q != rank]
        if idx:
            self.counts[rank][idx] = epoch

    # -------------------------------------------------------------- readback
    def status_words(self) -> np.ndarray:
        return self.status.cpu().numpy().view(np.uint32)

    def plan_host(self, rank: int) -> dict:
        p = self.plans[rank]
        m = int(p["m_total"].item())
        return dict(expert_offsets=p["expert_offsets"].cpu().numpy(),
                    src_info=p["src_info"][:m].cpu().numpy(),
                    seg_offsets=p["seg_offsets"].cpu().numpy(),
                    send_counts=p["send_counts"].cpu().numpy(),
                    gather_idx=p["gather_idx"][:m].cpu().numpy(), m_total=m)


def decode_trace(words: np.ndarray, n_blocks: int, records: int) -> list:
    """Per thread block: start time and one record per traced tile
    (tile, expert, completed_expert, t_ready, t_stored, t_done), times in ns."""
    stride = 2 + 4 * records
    out = []
    for b in range(n_blocks):
        w = words[b * stride:(b + 1) * stride]
        n = int(w[0])
        recs = []
        for i in range(min(n, records)):
            r = w[2 + 4 * i:6 + 4 * i]
            recs.append(dict(tile=int(r[0] & 0xFFFFFFFF), expert=int((r[0] >> 32) & 0x7FFFFFFF),
                             completed=bool(r[0] >> 63), t_ready=int(r[1]), t_stored=int(r[2]),
                             t_done=int(r[3])))
        out.append(dict(tiles=n, t_start=int(w[1]), records=recs))
    return out


def summarize_trace(tr: list) -> dict:
    """Where a fused launch spends its time, from a decoded trace."""
    starts = [b["t_start"] for b in tr if b["t_start"]]
    recs = [r for b in tr for r in b["records"]]
    if not starts or not recs:
        return {}
    t0 = min(starts)
    t1 = max(r["t_done"] for r in recs)
    epi = [r["t_stored"] - r["t_ready"] for r in recs]
    cnt = [r["t_done"] - r["t_stored"] for r in recs if not r["completed"]]
    sig = [r["t_done"] - r["t_stored"] for r in recs if r["completed"]]
    waits = []
    for b in tr:
        prev = b["t_start"]
        for r in b["records"]:
            waits.append(r["t_ready"] - prev)
            prev = r["t_done"]
    last_end = [max(r["t_done"] for r in b["records"]) - t0 for b in tr if b["records"]]

    def st(x):
        x = np.asarray(x, dtype=np.float64) / 1e3
        return {} if x.size == 0 else dict(n=int(x.size), mean_us=float(x.mean()),
                                           p50_us=float(np.median(x)), max_us=float(x.max()))
    return dict(span_us=(t1 - t0) / 1e3, tiles=len(recs), epilogue=st(epi), count=st(cnt),
                signal=st(sig), wait_for_accumulator=st(waits), block_end=st(last_end))
