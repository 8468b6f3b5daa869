"""Binding of the operators around the layer (``include/moe_block.h``): the
residual-add RMS norm and its backward, the 8-bit experts, the global gradient
norm and clipping. Same rules as the package: argument checks and marshalling
only, all arithmetic in the HIP kernels.

Codes and scales of 8-bit blocks are ``torch.uint8`` tensors, or
``torch.float8_e4m3fn`` codes with ``torch.float8_e8m0fnu`` scales (the same
bytes). Tensors have to lie on the current device.
"""
from __future__ import annotations

import ctypes
import operator

import expert_load_balance_amd as _moe

__all__ = [
    "moe_rmsnorm", "moe_rmsnorm_backward_workspace_bytes", "moe_rmsnorm_backward",
    "moe_mx_quantize", "moe_permute_mx", "moe_mx_workspace_bytes", "moe_grouped_gemm_mx",
    "moe_grad_workspace_bytes", "moe_grad_norm", "moe_grad_clip", "BLOCK_SYMBOLS", "MX_BLOCK",
]

#: entry points of include/moe_block.h
BLOCK_SYMBOLS = (
    "moe_rmsnorm", "moe_rmsnorm_backward_workspace_bytes", "moe_rmsnorm_backward",
    "moe_mx_quantize", "moe_permute_mx", "moe_mx_workspace_bytes", "moe_grouped_gemm_mx",
    "moe_grad_workspace_bytes", "moe_grad_norm", "moe_grad_clip",
)

#: values that share a scale
MX_BLOCK = 32

_VP = ctypes.c_void_p
_dtype_of = operator.attrgetter("dtype")


class GradT(ctypes.Structure):
    _fields_ = [("src", _VP), ("dst", _VP), ("count", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def signatures():
    """name -> (result type, argument types), for the package's load()."""
    st, sz, i32, i64, f32 = (ctypes.c_int, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64,
                             ctypes.c_float)
    sp, gp = ctypes.POINTER(_moe.Shape), ctypes.POINTER(GradT)
    return {
        "moe_rmsnorm": (st, [sp, _VP, _VP, _VP, f32, _VP, _VP, _VP, _VP, _VP, _VP]),
        "moe_rmsnorm_backward_workspace_bytes": (sz, [sp]),
        "moe_rmsnorm_backward": (st, [sp, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, sz, _VP]),
        "moe_mx_quantize": (st, [i64, i64, i32, _VP, _VP, _VP, _VP]),
        "moe_permute_mx": (st, [sp, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
        "moe_mx_workspace_bytes": (sz, [sp]),
        "moe_grouped_gemm_mx": (st, [sp, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, sz,
                                     _VP]),
        "moe_grad_workspace_bytes": (sz, [i32, gp]),
        "moe_grad_norm": (st, [i32, gp, _VP, _VP, _VP, sz, _VP]),
        "moe_grad_clip": (st, [i32, gp, f32, _VP, _VP]),
    }


_types = None


def _env():
    """(function giving the current device, activation types by moe_dtype, code
    types, scale types, float32, int32), looked up once: a call's own cost counts beside a decode step's kernels."""
    global _types
    if _types is None:
        import torch

        def device():
            try:
                return torch.cuda.current_device()
            except (RuntimeError, AssertionError):
                return -2  # no GPU: no tensor is there (host tensors are on -1)

        u8 = torch.uint8
        _types = (device, {_moe.MOE_F32: (torch.float32,), _moe.MOE_BF16: (torch.bfloat16,)},
                  (u8, torch.float8_e4m3fn), (u8, torch.float8_e8m0fnu), (torch.float32,), (torch.int32,))
    return _types


def _ptr(t, types, name, numel, here, nullable=False):
    """The package's pointer check, and that the tensor is where the launch
    is. The common case is one line; what fails it is told apart below."""
    if t is None and nullable:
        return None
    try:
        if (t.get_device() == here and t.is_contiguous() and t.numel() >= numel
                and (types is None or t.dtype in types)):
            return t.data_ptr() or None
    except AttributeError:
        pass
    _moe._ptr(t, types, name, numel, nullable)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{here}")


def _stream(stream, here):
    """The current device's current stream, or the one given."""
    if stream is None:
        import torch

        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # a Stream object costs more than the rest of the call
            return raw(here)
    return _moe._stream(stream)


def _mx(q, scales, name, n, here, nullable=False):
    """Pointers of codes and scales of n values."""
    _, _, ct, stp, _, _ = _env()
    return (_ptr(q, ct, name, n, here, nullable),
            _ptr(scales, stp, name + " scales", n // MX_BLOCK, here, nullable))


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def moe_rmsnorm(shape, x, weight, eps, residual=None, s=None, y=None, q=None, scales=None, rstd=None,
                stream=None):
    """s = x + residual; y and (q, scales) = s * rstd * weight. Outputs that are
    None are not computed; at least one is needed."""
    dev, acts, ct, stp, f32, _ = _env()
    here, T, H = dev(), shape.T, shape.H
    act, n = acts.get(shape.dtype), T * H
    st = _moe.load().moe_rmsnorm(
        ctypes.byref(shape), _ptr(x, act, "x", n, here), _ptr(residual, act, "residual", n, here, True),
        _ptr(weight, act, "weight", H, here), eps, _ptr(s, act, "s", n, here, True),
        _ptr(y, act, "y", n, here, True), _ptr(q, ct, "q", n, here, True),
        _ptr(scales, stp, "q scales", n // MX_BLOCK, here, True),
        _ptr(rstd, f32, "rstd", T, here, True), _stream(stream, here))
    _moe._ok(st, "moe_rmsnorm")


def moe_rmsnorm_backward_workspace_bytes(shape) -> int:
    return int(_moe.load().moe_rmsnorm_backward_workspace_bytes(ctypes.byref(shape)))


def moe_rmsnorm_backward(shape, s, weight, rstd, dy, dx, dweight, ws, ds=None, stream=None):
    """dx (of x and of residual alike; may be dy or ds) and dweight (float32)."""
    dev, acts, _, _, f32, _ = _env()
    here, T, H = dev(), shape.T, shape.H
    act, n = acts.get(shape.dtype), T * H
    st = _moe.load().moe_rmsnorm_backward(
        ctypes.byref(shape), _ptr(s, act, "s", n, here), _ptr(weight, act, "weight", H, here),
        _ptr(rstd, f32, "rstd", T, here), _ptr(dy, act, "dy", n, here), _ptr(ds, act, "ds", n, here, True),
        _ptr(dx, act, "dx", n, here), _ptr(dweight, f32, "dweight", H, here), _ptr(ws, None, "ws", 0, here),
        _bytes(ws), _stream(stream, here))
    _moe._ok(st, "moe_rmsnorm_backward")


def moe_mx_quantize(x, q, scales, stream=None):
    """x [..., cols] (bfloat16 or float32) in 8-bit blocks along its last dimension."""
    dev, acts, ct, stp, _, _ = _env()
    here = dev()
    if x.dim() < 1:
        raise ValueError("x needs a dimension to cut into blocks")
    n, cols = x.numel(), x.shape[-1]
    bf = x.dtype in acts[_moe.MOE_BF16]
    st = _moe.load().moe_mx_quantize(
        n // cols if cols else 0, cols, _moe.MOE_BF16 if bf else _moe.MOE_F32,
        _ptr(x, acts[_moe.MOE_BF16] + acts[_moe.MOE_F32], "x", 0, here), _ptr(q, ct, "q", n, here),
        _ptr(scales, stp, "q scales", n // MX_BLOCK, here), _stream(stream, here))
    _moe._ok(st, "moe_mx_quantize")


def moe_permute_mx(shape, q, scales, ids, eidx, plan, buf_q, buf_scales, dest_row, row_src, stream=None):
    """moe_permute for 8-bit rows."""
    dev, _, _, _, _, i32 = _env()
    here, N, H = dev(), shape.N, shape.H
    st = _moe.load().moe_permute_mx(
        ctypes.byref(shape), *_mx(q, scales, "q", shape.T * H, here), _ptr(ids, i32, "ids", N, here),
        _ptr(eidx, i32, "eidx", N, here), _ptr(plan, i32, "plan", _moe.plan_layout_total(shape), here),
        *_mx(buf_q, buf_scales, "buf_q", N * H, here), _ptr(dest_row, i32, "dest_row", N, here),
        _ptr(row_src, i32, "row_src", N, here), _stream(stream, here))
    _moe._ok(st, "moe_permute_mx")


def moe_mx_workspace_bytes(shape) -> int:
    return int(_moe.load().moe_mx_workspace_bytes(ctypes.byref(shape)))


def moe_grouped_gemm_mx(shape, a, a_scales, plan, w_gate, w_up, w_down, y, ws, stream=None):
    """moe_grouped_gemm on 8-bit blocks. w_gate, w_up, w_down: (codes, scales)
    of [E][F][H], [E][F][H] and [E][H][F]; y bfloat16 [N][H]."""
    dev, acts, _, _, _, i32 = _env()
    here, N, H = dev(), shape.N, shape.H
    n = shape.E * shape.F * H
    st = _moe.load().moe_grouped_gemm_mx(
        ctypes.byref(shape), *_mx(a, a_scales, "a", N * H, here),
        _ptr(plan, i32, "plan", _moe.plan_layout_total(shape), here), *_mx(*w_gate, "w_gate", n, here),
        *_mx(*w_up, "w_up", n, here), *_mx(*w_down, "w_down", n, here),
        _ptr(y, acts[_moe.MOE_BF16], "y", N * H, here), _ptr(ws, None, "ws", 0, here), _bytes(ws),
        _stream(stream, here))
    _moe._ok(st, "moe_grouped_gemm_mx")


def _columns(ts, other, here, what):
    """(addresses, element counts, moe_dtypes) of a list of gradients. The
    checks are the single pointer's, a column at a time: a step has hundreds of
    tensors."""
    import torch

    T = torch.Tensor
    _, acts, _, _, _, _ = _env()
    f32, bf = acts[_moe.MOE_F32][0], acts[_moe.MOE_BF16][0]
    try:  # mapped methods cost two thirds of a loop's
        dts = list(map(_dtype_of, ts))
        count = list(map(T.numel, ts))
        ok = (set(map(T.get_device, ts)) <= {here} and all(map(T.is_contiguous, ts))
              and set(dts) <= {f32, bf})
        if ok and other is not None:
            ok = dts == list(map(_dtype_of, other)) and count == list(map(T.numel, other))
    except (TypeError, AttributeError):
        ok = False
    if not ok:
        for i, t in enumerate(ts):
            _ptr(t, (f32, bf), f"{what} {i}", 0, here)
            if other is not None and (t.dtype != other[i].dtype or t.numel() != other[i].numel()):
                raise ValueError(f"{what} {i} differs from its gradient in type or size")
    return list(map(T.data_ptr, ts)), count, [_moe.MOE_BF16 if d is bf else _moe.MOE_F32 for d in dts]


def _grad_list(grads, into, here):
    """The moe_grad_t array of a list: four 64-bit words each (the last holds
    the type and a zero)."""
    n = len(grads)
    src, count, dtype = _columns(grads, None, here, "gradient")
    dst = src if into is None or into is grads else _columns(into, grads, here, "output")[0]
    words = [0] * (4 * n)
    words[0::4], words[1::4], words[2::4], words[3::4] = src, dst, count, dtype
    return ctypes.cast((ctypes.c_uint64 * (4 * n))(*words), ctypes.POINTER(GradT)) if n else None


def moe_grad_workspace_bytes(grads) -> int:
    """grads: the list of tensors that moe_grad_norm takes."""
    arr = (GradT * max(len(grads), 1))()
    for i, g in enumerate(grads):
        arr[i].count = g.numel()
    return int(_moe.load().moe_grad_workspace_bytes(len(grads), arr))


def moe_grad_norm(grads, norm, err, ws, stream=None):
    """norm (float32, one element) = the root of the sum of squares of all
    elements of a list of float32 and bfloat16 tensors; err (int32) gets
    ERR_NONFINITE when it is not finite."""
    dev, _, _, _, f32, i32 = _env()
    here = dev()
    st = _moe.load().moe_grad_norm(
        len(grads), _grad_list(grads, None, here), _ptr(norm, f32, "norm", 1, here),
        _ptr(err, i32, "err", 1, here), _ptr(ws, None, "ws", 0, here), _bytes(ws), _stream(stream, here))
    _moe._ok(st, "moe_grad_norm")


def moe_grad_clip(grads, into, max_norm, norm, stream=None):
    """into[i] = grads[i] * min(1, max_norm / norm); into may be grads."""
    dev, _, _, _, f32, _ = _env()
    here = dev()
    if len(into) != len(grads):
        raise ValueError(f"{len(grads)} gradients and {len(into)} outputs")
    st = _moe.load().moe_grad_clip(
        len(grads), _grad_list(grads, into, here), max_norm, _ptr(norm, f32, "norm", 1, here),
        _stream(stream, here))
    _moe._ok(st, "moe_grad_clip")
