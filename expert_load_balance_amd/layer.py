"""Buffers and call sequence for one MoE layer forward on the GPU.

Plumbing only: torch allocates the device buffers once per shape (static
shapes: nothing here depends on the routing), and ``forward`` calls the C
entry points in the layer's order on one stream. No arithmetic happens in
Python.
"""
from __future__ import annotations

import torch

from . import (MOE_BF16, MOE_W_BF16, MOE_W_MX4, MOE_W_MX8, MX_BLOCK, Shape, moe_combine, moe_count_plan,
               moe_few_layer, moe_few_workspace_bytes, moe_gemm_down, moe_gemm_gateup, moe_gemm_schedule, moe_grouped_gemm_mx, moe_grouped_gemm_mx4,
               moe_grouped_gemm_slots,
               moe_grouped_gemm_train, moe_mx4_workspace_bytes, moe_mx_workspace_bytes, moe_permute, moe_permute_mx, moe_plan,
               moe_plan_layout, moe_prefetch_replicas, moe_rmsnorm, moe_route, moe_router,
               moe_router_workspace_bytes, moe_workspace_bytes)

STAGES = ("route", "count_plan", "permute", "gemm_schedule", "gemm_gateup", "gemm_down",
          "shared", "combine")


def alloc(shape, dtype, device):
    """torch.empty that never hands out a null pointer (empty shapes keep a
    one-element allocation behind a zero-length view)."""
    n = 1
    for d in shape:
        n *= d
    return torch.empty(max(n, 1), dtype=dtype, device=device)[:n].view(shape)


def _check_here(*tensors):
    """The layer's kernels run on the current device; the calls that come first
    do not look where their tensors are."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"a tensor of the layer is on {t.device}, the current device is cuda:{here}")


def _torch_stream(stream):
    """torch's object for a stream or its handle (an ExternalStream of handle 0
    would be a new stream)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()


class MoeLayerBuffers:
    """Every buffer of one layer call, sized by the shape alone.

    shared_F: width of an always-on shared expert (None: no shared expert).
    """

    def __init__(self, shape: Shape, device="cuda", shared_F: int | None = None):
        self.shape = shape
        T, H, E, k, R = shape.T, shape.H, shape.E, shape.k, shape.R
        N = T * k
        act = torch.bfloat16 if shape.dtype == MOE_BF16 else torch.float32
        i32 = torch.int32
        self.ids = alloc((T, k), i32, device)
        self.w = alloc((T, k), torch.float32, device)
        self.err = torch.zeros(1, dtype=i32, device=device)
        self.counts = alloc((E,), i32, device)
        self.offsets = alloc((E + 1,), i32, device)
        self.eidx = alloc((N,), i32, device)
        self.rank_load = alloc((R,), i32, device)
        self.plan = alloc((moe_plan_layout(shape)["total"],), i32, device)
        self.buf = alloc((N, H), act, device)
        self.dest_row = alloc((T, k), i32, device)
        self.row_src = alloc((N,), i32, device)
        self.y = alloc((N, H), act, device)
        self.out = alloc((T, H), act, device)
        self.ws = torch.empty(max(moe_workspace_bytes(shape), 256), dtype=torch.uint8, device=device)
        self.shared_shape = None
        if shared_F is not None:
            # one expert, one rank, k = 1: the plan is a single piece of T rows
            self.shared_shape = Shape(T, H, 1, 1, shared_F, 1, 0, shape.dtype)
            self.shared_counts = torch.full((1,), T, dtype=i32, device=device)
            self.shared_plan = alloc((moe_plan_layout(self.shared_shape)["total"],), i32, device)
            self.shared_ws = torch.empty(max(moe_workspace_bytes(self.shared_shape), 256),
                                         dtype=torch.uint8, device=device)
            self.shared_y = alloc((T, H), act, device)
            moe_plan(self.shared_shape, self.shared_counts, self.shared_plan)

    def forward(self, logits, bias, x, w_gate, w_up, w_down, shared_w=None, stream=None,
                marks=None, pool=None, gu=None):
        """Route -> count + plan (one launch up to 16384 assignments) -> permute ->
        grouped GEMM -> (shared) -> combine.

        marks: optional dict stage -> (start_event, end_event) recorded around
        each stage on the stream ("gemm" spans the routed grouped GEMM's three
        calls: schedule, gate/up, down). pool: a device buffer of
        moe_pool_bytes(shape) bytes; with it the planned replicas are
        prefetched into their slots after the plan and the grouped GEMM runs
        by plan segment, reading them (stages "prefetch" and "gemm_slots").
        gu: a bf16 [N, 2F] buffer; with it the grouped GEMM also keeps g | u
        for the backward (stage "gemm_train"). Returns self.out."""
        s = self.shape
        st = stream if stream is not None else torch.cuda.current_stream()

        def mark(name, i):
            if marks is not None and name in marks:
                marks[name][i].record(st)

        self.err.zero_()
        mark("route", 0)
        moe_route(s, logits, bias, self.ids, self.w, self.err, st)
        mark("route", 1)
        mark("count_plan", 0)
        moe_count_plan(s, self.ids, self.counts, self.offsets, self.eidx, self.rank_load, self.err,
                       self.ws, self.plan, st)
        mark("count_plan", 1)
        if pool is not None:
            mark("prefetch", 0)
            moe_prefetch_replicas(s, self.plan, w_gate, w_up, w_down, pool, st)
            mark("prefetch", 1)
        mark("permute", 0)
        moe_permute(s, x, self.ids, self.eidx, self.plan, self.buf, self.dest_row, self.row_src, st)
        mark("permute", 1)
        if gu is not None:
            mark("gemm_train", 0)
            moe_grouped_gemm_train(s, self.buf, self.plan, w_gate, w_up, w_down, self.y, gu,
                                   self.ws, st)
            mark("gemm_train", 1)
        elif pool is not None:
            mark("gemm_slots", 0)
            moe_grouped_gemm_slots(s, self.buf, self.plan, w_gate, w_up, w_down, pool, self.y,
                                   self.ws, st)
            mark("gemm_slots", 1)
        else:
            mark("gemm", 0)
            mark("gemm_schedule", 0)
            moe_gemm_schedule(s, self.plan, self.ws, st)
            mark("gemm_schedule", 1)
            mark("gemm_gateup", 0)
            moe_gemm_gateup(s, self.buf, self.plan, w_gate, w_up, self.ws, st)
            mark("gemm_gateup", 1)
            mark("gemm_down", 0)
            moe_gemm_down(s, self.plan, w_down, self.y, self.ws, st)
            mark("gemm_down", 1)
            mark("gemm", 1)
        shared_y = None
        if self.shared_shape is not None and shared_w is not None:
            mark("shared", 0)
            sg, su, sd = shared_w
            moe_gemm_schedule(self.shared_shape, self.shared_plan, self.shared_ws, st)
            moe_gemm_gateup(self.shared_shape, x, self.shared_plan, sg, su, self.shared_ws, st)
            moe_gemm_down(self.shared_shape, self.shared_plan, sd, self.shared_y, self.shared_ws, st)
            mark("shared", 1)
            shared_y = self.shared_y
        mark("combine", 0)
        moe_combine(s, self.y, self.dest_row, self.w, shared_y, self.out, st)
        mark("combine", 1)
        return self.out


class MoeLayerMx:
    """Buffers and call sequence of a serving step: norm (with the residual's
    addition), router, and the experts in 8-bit blocks.

    A shape whose dtype is MOE_BF16 with H and F multiples of 128. Weights are
    (codes, scales) pairs as moe_mx_quantize makes them, or, with weight_bits 4, as
    moe_mx4_quantize does (rows and activations stay in 8 bits). The buffers belong to
    one call at a time: calls that may overlap take an object each. A layer with a
    shared expert makes forward's calls itself and hands that expert's rows, made
    from self.xn, to experts.
    """

    def __init__(self, shape: Shape, device="cuda", weight_bits: int = 8):
        if weight_bits not in (4, 8):
            raise ValueError(f"weights of {weight_bits} bits: 8 or 4")
        self.shape, self.weight_bits = shape, weight_bits
        T, H, E, k, R = shape.T, shape.H, shape.E, shape.k, shape.R
        N, i32, u8, f32 = T * k, torch.int32, torch.uint8, torch.float32
        self.s = alloc((T, H), torch.bfloat16, device)
        self.xn = alloc((T, H), torch.bfloat16, device)
        self.xq = alloc((T, H), u8, device)
        self.xs = alloc((T, H // MX_BLOCK), u8, device)
        self.logits = alloc((T, E), f32, device)
        self.ids = alloc((T, k), i32, device)
        self.w = alloc((T, k), f32, device)
        self.err = torch.zeros(1, dtype=i32, device=device)
        self.counts = alloc((E,), i32, device)
        self.offsets = alloc((E + 1,), i32, device)
        self.eidx = alloc((N,), i32, device)
        self.rank_load = alloc((R,), i32, device)
        self.plan = alloc((moe_plan_layout(shape)["total"],), i32, device)
        self.buf_q = alloc((N, H), u8, device)
        self.buf_s = alloc((N, H // MX_BLOCK), u8, device)
        self.dest_row = alloc((T, k), i32, device)
        self.row_src = alloc((N,), i32, device)
        self.y = alloc((N, H), torch.bfloat16, device)
        self.out = alloc((T, H), torch.bfloat16, device)

        def bytes_(n):
            return torch.empty(max(n, 256), dtype=u8, device=device)

        # the bf16 layer's workspace also holds partial tiles of its GEMM; the
        # count needs only the head of it, but its size is one per shape
        self.ws = bytes_(moe_workspace_bytes(shape))
        self.router_ws = bytes_(moe_router_workspace_bytes(shape))
        self.mx_ws = bytes_((moe_mx_workspace_bytes if weight_bits == 8 else moe_mx4_workspace_bytes)(shape))

    def experts(self, xq, xs, ids, w, w_gate, w_up, w_down, shared_y=None, stream=None):
        """Count + plan, dispatch, the grouped GEMM on blocks and the combine, from
        the 8-bit rows and the router's choice (ids, gate weights w) to
        self.out."""
        s, st = self.shape, stream if stream is not None else torch.cuda.current_stream()
        _check_here(self.err, ids, w, shared_y)
        moe_count_plan(s, ids, self.counts, self.offsets, self.eidx, self.rank_load, self.err,
                       self.ws, self.plan, st)
        moe_permute_mx(s, xq, xs, ids, self.eidx, self.plan, self.buf_q, self.buf_s, self.dest_row,
                       self.row_src, st)
        gemm = moe_grouped_gemm_mx if self.weight_bits == 8 else moe_grouped_gemm_mx4
        gemm(s, self.buf_q, self.buf_s, self.plan, w_gate, w_up, w_down, self.y, self.mx_ws, st)
        moe_combine(s, self.y, self.dest_row, w, shared_y, self.out, st)
        return self.out

    def forward(self, x, residual, norm_weight, eps, w_router, bias, w_gate, w_up, w_down,
                stream=None):
        """One step: returns (out, s), the experts' sum and the residual stream
        x + residual that it is to be added to (the next norm's residual)."""
        st = stream if stream is not None else torch.cuda.current_stream()
        _check_here(self.err, w_router, bias)
        with torch.cuda.stream(_torch_stream(st)):
            self.err.zero_()
        moe_rmsnorm(self.shape, x, norm_weight, eps, residual=residual, s=self.s, y=self.xn,
                    q=self.xq, scales=self.xs, stream=st)
        moe_router(self.shape, self.xn, w_router, bias, self.logits, self.ids, self.w, self.err,
                   self.router_ws, st)
        self.experts(self.xq, self.xs, self.ids, self.w, w_gate, w_up, w_down, stream=st)
        return self.out, self.s


class MoeLayerFew:
    """Buffers and the call of a decode step of up to FEW_TOKENS tokens: router,
    top-k, experts and combine in moe_few_layer.

    A bf16 shape; weights: "bf16", "mx8" or "mx4", the form of every projection;
    shared_F: width of an always-on shared expert of the same form (None: no shared
    expert). The buffers belong to one call at a time: calls that may overlap, and
    captured graphs that may, take an object each. On 4-bit weights MoeLayerMx can be
    faster where more than 16 tokens choose and an expert has more than 12 of them on
    average (by a fifth at 32 tokens that choose every expert).
    """

    FORMS = {"bf16": MOE_W_BF16, "mx8": MOE_W_MX8, "mx4": MOE_W_MX4}

    def __init__(self, shape: Shape, device="cuda", weights="mx8", shared_F: int | None = None):
        self.shape, self.form, self.shared_F = shape, self.FORMS[weights], shared_F or 0
        T, k = shape.T, shape.k
        need = moe_few_workspace_bytes(shape, self.form, self.shared_F)
        if need == 0:
            raise ValueError(f"moe_few_layer has no layer of this shape on {weights} weights")
        self.out = alloc((T, shape.H), torch.bfloat16, device)
        self.ids = alloc((T, k), torch.int32, device)
        self.w = alloc((T, k), torch.float32, device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device)

    def forward(self, x, w_router, bias, w_gate, w_up, w_down, shared_w=None, stream=None):
        """Returns self.out; the router's choice is in self.ids and self.w, and
        self.err gathers MOE_ERR_NONFINITE from call to call. Weights are (values,
        scales) pairs, scales None in bfloat16; shared_w: the shared expert's three."""
        moe_few_layer(self.shape, self.form, x, w_router, bias, w_gate, w_up, w_down, self.out, self.err, self.ws,
                      shared=shared_w, shared_F=self.shared_F, ids=self.ids, w=self.w, stream=stream)
        return self.out
