"""include/moe_block.h without a GPU: every declared entry point is exported
and bound, and bad arguments are refused on the host before any launch."""
import ctypes
import os
import re

import pytest

import expert_load_balance_amd as moe
from expert_load_balance_amd.block import GradT

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUP = 1, 2
V = ctypes.c_void_p
P = V(4096)   # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        pytest.fail("libmoe.so is not built: run `python -m expert_load_balance_amd.build`")
    return moe.load()


def test_declared_symbols_are_exported_and_bound(lib):
    with open(os.path.join(ROOT, "include", "moe_block.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text)))
    assert names == sorted(moe.BLOCK_SYMBOLS)
    for n in names:
        assert hasattr(lib, n) and callable(getattr(moe, n)), n


def test_plan_layout_total_follows_the_layout(lib):
    for T, E, k, R in [(16, 8, 2, 4), (1, 1, 1, 1), (300, 36, 5, 12), (8, 256, 8, 64), (9, 255, 3, 51)]:
        s = moe.Shape(T, 128, E, k, 128, R, 1)
        assert moe.plan_layout_total(s) == moe.moe_plan_layout(s)["total"]


def _norm(lib, s, x=P, r=None, w=P, eps=1e-6, so=None, y=P, q=None, sc=None, rstd=None):
    return lib.moe_rmsnorm(ctypes.byref(s), x, r, w, eps, so, y, q, sc, rstd, None)


def test_rmsnorm_refusals(lib):
    s = moe.Shape(16, 64, 8, 2, 128, 4, 2, moe.MOE_F32)
    assert _norm(lib, s.replace(T=-1)) == EINVAL
    assert _norm(lib, s, x=None) == EINVAL
    assert _norm(lib, s, w=None) == EINVAL
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(lib, s, eps=eps) == EINVAL, eps
    assert _norm(lib, s, y=None) == EINVAL                    # nothing to compute
    assert _norm(lib, s, q=P) == EINVAL                       # codes without scales
    assert _norm(lib, s, sc=P) == EINVAL
    assert _norm(lib, s, so=P, y=P) == EINVAL                 # both outputs in one place
    assert _norm(lib, s.replace(H=68), q=P, sc=P) == EUNSUP   # blocks of 32 do not fit
    for name in ("x", "r", "w", "so", "y"):
        assert _norm(lib, s, **{name: V(4096 + 8)}) == EINVAL, name   # misaligned
    assert _norm(lib, s, rstd=V(4098)) == EINVAL
    assert _norm(lib, s.replace(T=0), x=None, y=None) == 0    # no rows: nothing to launch


def test_rmsnorm_backward_refusals(lib):
    s = moe.Shape(16, 64, 8, 2, 128, 4, 2, moe.MOE_BF16)
    need = moe.moe_rmsnorm_backward_workspace_bytes(s)
    assert need >= 16 * 64 * 4 and moe.moe_rmsnorm_backward_workspace_bytes(s.replace(R=3)) == 0
    good = [P, P, P, P, None, P, P, P, need, None]            # s w rstd dy ds dx dw ws bytes stream
    f = lib.moe_rmsnorm_backward
    for i in (0, 1, 2, 3, 5, 6, 7):
        a = list(good)
        a[i] = None
        assert f(ctypes.byref(s), *a) == EINVAL, i
        a[i] = V(4097)
        assert f(ctypes.byref(s), *a) == EINVAL, i
    a = list(good)
    a[8] = need - 1
    assert f(ctypes.byref(s), *a) == EINVAL
    assert f(ctypes.byref(s.replace(E=0)), *good) == EINVAL


def test_quantize_refusals(lib):
    f = lib.moe_mx_quantize
    assert f(-1, 64, moe.MOE_BF16, P, P, P, None) == EINVAL
    assert f(4, 0, moe.MOE_BF16, P, P, P, None) == EINVAL
    assert f(4, 64, 7, P, P, P, None) == EINVAL
    assert f(4, 48, moe.MOE_BF16, P, P, P, None) == EUNSUP
    assert f(1 << 35, 64, moe.MOE_BF16, P, P, P, None) == EINVAL
    assert f(1 << 62, 1 << 10, moe.MOE_BF16, P, P, P, None) == EINVAL   # the product would wrap
    for i in range(3):
        a = [P, P, P]
        a[i] = None
        assert f(4, 64, moe.MOE_F32, *a, None) == EINVAL
        a[i] = V(4100)
        assert f(4, 64, moe.MOE_F32, *a, None) == EINVAL
    assert f(0, 64, moe.MOE_F32, None, None, None, None) == 0


def test_mx_layer_refusals(lib):
    s = moe.Shape(16, 128, 8, 2, 128, 4, 2, moe.MOE_BF16)
    need = moe.moe_mx_workspace_bytes(s)
    assert need >= 32 * 128 + 32 * 4
    assert moe.moe_mx_workspace_bytes(s.replace(H=192)) == 0
    f, n = lib.moe_permute_mx, 9
    assert f(ctypes.byref(s.replace(dtype=moe.MOE_F32)), *[P] * n, None) == EUNSUP
    assert f(ctypes.byref(s.replace(F=192)), *[P] * n, None) == EUNSUP
    assert f(ctypes.byref(s.replace(R=3)), *[P] * n, None) == EINVAL
    for i in range(n):
        a = [P] * n
        a[i] = None
        assert f(ctypes.byref(s), *a, None) == EINVAL, i
    g = lib.moe_grouped_gemm_mx
    for i in range(11):
        a = [P] * 11
        a[i] = None
        assert g(ctypes.byref(s), *a, need, None) == EINVAL, i
        if i != 2:                                            # (the plan is int32: 4-byte aligned)
            a[i] = V(4096 + 8)
            assert g(ctypes.byref(s), *a, need, None) == EINVAL, i
    assert g(ctypes.byref(s), *[P] * 11, need - 1, None) == EINVAL
    assert g(ctypes.byref(s.replace(H=64)), *[P] * 11, need, None) == EUNSUP


def _grads(*items):
    arr = (GradT * max(len(items), 1))()
    for i, (src, dst, count, dtype) in enumerate(items):
        arr[i].src, arr[i].dst, arr[i].count, arr[i].dtype = src, dst, count, dtype
    return arr


def test_grad_refusals(lib):
    ok = _grads((4096, 4096, 100, moe.MOE_F32), (None, None, 0, moe.MOE_BF16))
    need = lib.moe_grad_workspace_bytes(2, ok)
    assert need > 0 and lib.moe_grad_workspace_bytes(0, None) > 0
    assert lib.moe_grad_workspace_bytes(-1, ok) == 0
    assert lib.moe_grad_workspace_bytes(1, None) == 0
    norm, clip = lib.moe_grad_norm, lib.moe_grad_clip
    for item in [(4096, 4096, -1, 0), (4096, 4096, 1 << 40, 0), (4096, 4096, 4, 5), (None, 4096, 4, 0),
                 (4098, 4096, 4, moe.MOE_F32), (4097, 4096, 4, moe.MOE_BF16)]:
        assert norm(1, _grads(item), P, P, P, need, None) == EINVAL, item
        assert clip(1, _grads(item), 1.0, P, None) == EINVAL, item
    for a in [(None, P, P, need), (P, None, P, need), (P, P, None, need), (P, P, P, 0), (P, P, V(4100), need)]:
        assert norm(2, ok, *a, None) == EINVAL
    assert norm(-1, ok, P, P, P, need, None) == EINVAL
    assert clip(1, _grads((4096, None, 4, 0)), 1.0, P, None) == EINVAL
    for m in (-1.0, float("nan"), float("inf")):
        assert clip(2, ok, m, P, None) == EINVAL
    assert clip(2, ok, 1.0, None, None) == EINVAL


@pytest.mark.parametrize("items", [
    [(4096, 4096, 64, 0), (4096, 4096, 64, 0)],          # one tensor twice, in place
    [(4096, 8192, 64, 0), (20480, 8192, 64, 0)],         # two into one
    [(4096, 4100, 64, 0)],                               # its own source in part
    [(4096, 8192, 64, 0), (8192 + 128, 16384, 64, 0)],   # one's output in another's source
    [(8192 + 128, 16384, 8, 0), (4096, 8192, 64, 0)],
    [(4096, 32768, 4096, 0), (20484, 20484, 8, 0), (4096 + 512, 65536, 16, 0), (40960, 40960, 4, 1)],
], ids=["twice", "two_into_one", "own_part", "into_source", "into_source_back", "nested"])
def test_clip_refuses_overlaps(lib, items):
    assert lib.moe_grad_clip(len(items), _grads(*items), 1.0, P, None) == EINVAL


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    s = moe.Shape(4, 64, 8, 2, 128, 4, 2, moe.MOE_F32)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.moe_rmsnorm(s, x, x[0], 1e-6, y=x)
    with pytest.raises(ValueError):
        moe.moe_mx_quantize(x, x.to(torch.uint8), x.to(torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_grad_norm([x], x, x, x)
    with pytest.raises(ValueError):
        moe.moe_grad_clip([x], [], 1.0, x)
