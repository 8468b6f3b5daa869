"""Binding of ``include/moe_step.h``: the norms between two blocks of a residual
stream and their backward, 4-bit blocks and the experts on them, the layer for a
few tokens. Same rules as ``block.py``: argument checks and marshalling only;
tensors have to lie on the current device.

4-bit codes are ``torch.uint8`` tensors (two codes a byte) or
``torch.float4_e2m1fn_x2``; scales ``torch.uint8`` or ``torch.float8_e8m0fnu``.
"""
from __future__ import annotations

import ctypes

import expert_load_balance_amd as _moe

from .block import MX_BLOCK, _bytes, _env, _ptr, _stream

__all__ = [
    "moe_block_norm", "moe_block_norm_backward_workspace_bytes", "moe_block_norm_backward",
    "moe_mx4_quantize", "moe_mx4_dequantize", "moe_mx4_workspace_bytes", "moe_grouped_gemm_mx4",
    "moe_few_workspace_bytes", "moe_few_layer", "STEP_SYMBOLS",
    "MOE_W_BF16", "MOE_W_MX8", "MOE_W_MX4", "FEW_TOKENS",
]

#: entry points of include/moe_step.h
STEP_SYMBOLS = (
    "moe_block_norm", "moe_block_norm_backward_workspace_bytes", "moe_block_norm_backward",
    "moe_mx4_quantize", "moe_mx4_dequantize", "moe_mx4_workspace_bytes", "moe_grouped_gemm_mx4",
    "moe_few_workspace_bytes", "moe_few_layer",
)

#: forms of moe_few_layer's weights, and its most tokens
MOE_W_BF16, MOE_W_MX8, MOE_W_MX4 = 0, 1, 2
FEW_TOKENS = 32

_VP = ctypes.c_void_p


class FewWeightsT(ctypes.Structure):
    _fields_ = [(n, _VP) for n in ("gate", "up", "down", "gate_scales", "up_scales", "down_scales")]


def signatures():
    """name -> (result type, argument types), for the package's load()."""
    st, sz, i32, i64, f32 = (ctypes.c_int, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64,
                             ctypes.c_float)
    sp, wp = ctypes.POINTER(_moe.Shape), ctypes.POINTER(FewWeightsT)
    return {
        "moe_block_norm": (st, [sp, _VP, _VP, f32, _VP, _VP, i32, _VP, f32, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
        "moe_block_norm_backward_workspace_bytes": (sz, [sp, i32]),
        "moe_block_norm_backward": (st, [sp, _VP, _VP, _VP, _VP, f32, _VP, _VP, i32, _VP, _VP, _VP, _VP, _VP, _VP,
                                         _VP, _VP, _VP, sz, _VP]),
        "moe_mx4_quantize": (st, [i64, i64, i32, _VP, _VP, _VP, _VP]),
        "moe_mx4_dequantize": (st, [i64, i64, i32, _VP, _VP, _VP, _VP]),
        "moe_mx4_workspace_bytes": (sz, [sp]),
        "moe_grouped_gemm_mx4": (st, [sp, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, sz, _VP]),
        "moe_few_workspace_bytes": (sz, [sp, i32, i32]),
        "moe_few_layer": (st, [sp, i32, _VP, _VP, _VP, wp, wp, i32, _VP, _VP, _VP, _VP, _VP, sz, _VP]),
    }


_codes = None


def _fours():
    """Types of 4-bit codes."""
    global _codes
    if _codes is None:
        import torch

        four = getattr(torch, "float4_e2m1fn_x2", None)
        _codes = (torch.uint8,) if four is None else (torch.uint8, four)
    return _codes


def _gate_values(shape, gate_rows):
    """Elements of a gate and of its gradient."""
    return shape.T if gate_rows == 0 else -(-shape.T // gate_rows) * shape.H if gate_rows > 0 else 0


def moe_block_norm(shape, x, eps, residual=None, alpha=1.0, w_post=None, gate=None, gate_rows=0, w_pre=None, s=None,
                   y=None, q=None, scales=None, rstd_post=None, rstd_pre=None, stream=None):
    """s = alpha * residual + gate * norm(x, w_post); y and (q, scales) = norm(s,
    w_pre). gate: one value a token (gate_rows 0), or a row of H for every
    gate_rows tokens. Outputs that are None are not computed; at least one is
    needed."""
    dev, acts, ct, stp, f32, _ = _env()
    here, T, H = dev(), shape.T, shape.H
    act, n = acts.get(shape.dtype), T * H
    st = _moe.load().moe_block_norm(
        ctypes.byref(shape), _ptr(x, act, "x", n, here), _ptr(residual, act, "residual", n, here, True), alpha,
        _ptr(w_post, act, "w_post", H, here, True), _ptr(gate, act, "gate", _gate_values(shape, gate_rows), here, True),
        gate_rows, _ptr(w_pre, act, "w_pre", H, here, True), eps, _ptr(s, act, "s", n, here, True),
        _ptr(y, act, "y", n, here, True), _ptr(q, ct, "q", n, here, True),
        _ptr(scales, stp, "q scales", n // MX_BLOCK, here, True), _ptr(rstd_post, f32, "rstd_post", T, here, True),
        _ptr(rstd_pre, f32, "rstd_pre", T, here, True), _stream(stream, here))
    _moe._ok(st, "moe_block_norm")


def moe_block_norm_backward_workspace_bytes(shape, gate_rows=0) -> int:
    return int(_moe.load().moe_block_norm_backward_workspace_bytes(ctypes.byref(shape), gate_rows))


def moe_block_norm_backward(shape, x, rstd_post, dy, ds, dx, ws, s=None, rstd_pre=None, alpha=1.0, w_post=None,
                            gate=None, gate_rows=0, w_pre=None, dresidual=None, dw_post=None, dgate=None, dw_pre=None,
                            stream=None):
    """dx, and those of dresidual, dw_post, dgate and dw_pre (float32) that are
    not None. dy is the gradient of y, ds the one that reaches s past the norm
    (one may be None)."""
    dev, acts, _, _, f32, _ = _env()
    here, T, H = dev(), shape.T, shape.H
    act, n, gates = acts.get(shape.dtype), T * H, _gate_values(shape, gate_rows)
    st = _moe.load().moe_block_norm_backward(
        ctypes.byref(shape), _ptr(x, act, "x", n, here), _ptr(rstd_post, f32, "rstd_post", T, here, True),
        _ptr(s, act, "s", n, here, True), _ptr(rstd_pre, f32, "rstd_pre", T, here, True), alpha,
        _ptr(w_post, act, "w_post", H, here, True), _ptr(gate, act, "gate", gates, here, True), gate_rows,
        _ptr(w_pre, act, "w_pre", H, here, True), _ptr(dy, act, "dy", n, here, True), _ptr(ds, act, "ds", n, here, True),
        _ptr(dx, act, "dx", n, here), _ptr(dresidual, act, "dresidual", n, here, True),
        _ptr(dw_post, f32, "dw_post", H, here, True), _ptr(dgate, f32, "dgate", gates, here, True),
        _ptr(dw_pre, f32, "dw_pre", H, here, True), _ptr(ws, None, "ws", 0, here), _bytes(ws), _stream(stream, here))
    _moe._ok(st, "moe_block_norm_backward")


def _matrix(x):
    """(rows, columns, moe_dtype) of a tensor in blocks along its last dimension."""
    if x.dim() < 1:
        raise ValueError("x needs a dimension to cut into blocks")
    _, acts, _, _, _, _ = _env()
    n, cols = x.numel(), x.shape[-1]
    return n // cols if cols else 0, cols, _moe.MOE_BF16 if x.dtype in acts[_moe.MOE_BF16] else _moe.MOE_F32


def moe_mx4_quantize(x, q, scales, stream=None):
    """x [..., cols] (bfloat16 or float32) in 4-bit blocks along its last dimension."""
    dev, acts, _, stp, _, _ = _env()
    here, n = dev(), x.numel()
    rows, cols, dtype = _matrix(x)
    st = _moe.load().moe_mx4_quantize(
        rows, cols, dtype, _ptr(x, acts[_moe.MOE_BF16] + acts[_moe.MOE_F32], "x", 0, here),
        _ptr(q, _fours(), "q", n // 2, here), _ptr(scales, stp, "q scales", n // MX_BLOCK, here), _stream(stream, here))
    _moe._ok(st, "moe_mx4_quantize")


def moe_mx4_dequantize(q, scales, x, stream=None):
    """The values of 4-bit blocks, into x [..., cols] (bfloat16 or float32)."""
    dev, acts, _, stp, _, _ = _env()
    here, n = dev(), x.numel()
    rows, cols, dtype = _matrix(x)
    st = _moe.load().moe_mx4_dequantize(
        rows, cols, dtype, _ptr(q, _fours(), "q", n // 2, here), _ptr(scales, stp, "q scales", n // MX_BLOCK, here),
        _ptr(x, acts[_moe.MOE_BF16] + acts[_moe.MOE_F32], "x", 0, here), _stream(stream, here))
    _moe._ok(st, "moe_mx4_dequantize")


def moe_mx4_workspace_bytes(shape) -> int:
    return int(_moe.load().moe_mx4_workspace_bytes(ctypes.byref(shape)))


def moe_grouped_gemm_mx4(shape, a, a_scales, plan, w_gate, w_up, w_down, y, ws, stream=None):
    """moe_grouped_gemm_mx with weights in 4-bit blocks. w_gate, w_up, w_down:
    (codes, scales) of [E][F][H], [E][F][H] and [E][H][F] values; y bfloat16 [N][H]."""
    dev, acts, ct, stp, _, i32 = _env()
    here, N, H = dev(), shape.N, shape.H
    n, four = shape.E * shape.F * H, _fours()
    w = []
    for name, (q, s) in zip(("w_gate", "w_up", "w_down"), (w_gate, w_up, w_down)):
        w += [_ptr(q, four, name, n // 2, here), _ptr(s, stp, name + " scales", n // MX_BLOCK, here)]
    st = _moe.load().moe_grouped_gemm_mx4(
        ctypes.byref(shape), _ptr(a, ct, "a", N * H, here), _ptr(a_scales, stp, "a scales", N * H // MX_BLOCK, here),
        _ptr(plan, i32, "plan", _moe.plan_layout_total(shape), here), *w,
        _ptr(y, acts[_moe.MOE_BF16], "y", N * H, here), _ptr(ws, None, "ws", 0, here), _bytes(ws), _stream(stream, here))
    _moe._ok(st, "moe_grouped_gemm_mx4")


def moe_few_workspace_bytes(shape, form, shared_F=0) -> int:
    return int(_moe.load().moe_few_workspace_bytes(ctypes.byref(shape), form, shared_F))


def _few_weights(form, projections, n, here, what):
    """The struct of (values, scales) of gate, up and down, each of n values."""
    _, acts, ct, stp, _, _ = _env()
    out = FewWeightsT()
    for name, (v, s) in zip(("gate", "up", "down"), projections):
        name_ = f"{what} {name}"
        if form == MOE_W_BF16:
            setattr(out, name, _ptr(v, acts[_moe.MOE_BF16], name_, n, here))
        else:
            setattr(out, name, _ptr(v, ct if form == MOE_W_MX8 else _fours(), name_, n if form == MOE_W_MX8 else n // 2, here))
            setattr(out, name + "_scales", _ptr(s, stp, name_ + " scales", n // MX_BLOCK, here))
    return out


def moe_few_layer(shape, form, x, w_router, bias, gate, up, down, out, err, ws, shared=None, shared_F=0, ids=None, w=None,
                  stream=None):
    """Router, top-k, experts, shared expert and combine of up to FEW_TOKENS
    tokens. gate, up, down: (values, scales) of [E][F][H], [E][F][H] and
    [E][H][F], scales None in bfloat16; shared: the three of one expert of width
    shared_F; ids and w, the router's choice, may be None."""
    dev, acts, _, _, f32, i32 = _env()
    here, T, H, E = dev(), shape.T, shape.H, shape.E
    bf = acts[_moe.MOE_BF16]
    routed = _few_weights(form, (gate, up, down), E * shape.F * H, here, "routed")
    one = None if shared is None else _few_weights(form, shared, shared_F * H, here, "shared")
    st = _moe.load().moe_few_layer(
        ctypes.byref(shape), form, _ptr(x, bf, "x", T * H, here), _ptr(w_router, bf, "w_router", E * H, here),
        _ptr(bias, f32, "bias", E, here, True), ctypes.byref(routed), None if one is None else ctypes.byref(one), shared_F,
        _ptr(out, bf, "out", T * H, here), _ptr(ids, i32, "ids", shape.N, here, True), _ptr(w, f32, "w", shape.N, here, True),
        _ptr(err, i32, "err", 1, here), _ptr(ws, None, "ws", 0, here), _bytes(ws), _stream(stream, here))
    _moe._ok(st, "moe_few_layer")
