"""include/moe_step.h without a GPU: every declared entry point is exported and
bound, bad arguments are refused on the host before any launch, and the float64
forms that the GPU tests go by are right."""
import ctypes
import os
import re

import pytest

import expert_load_balance_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUP = 1, 2
V = ctypes.c_void_p
P = V(4096)   # aligned, never dereferenced: validation fails first
NORM = moe.Shape(16, 64, 8, 2, 128, 4, 2, moe.MOE_BF16)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        pytest.fail("libmoe.so is not built: run `python -m expert_load_balance_amd.build`")
    return moe.load()


def test_declared_symbols_are_exported_and_bound(lib):
    with open(os.path.join(ROOT, "include", "moe_step.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(moe.STEP_SYMBOLS)
    for n in names:
        assert hasattr(lib, n) and callable(getattr(moe, n)), n


def _fwd(lib, s=NORM, x=P, r=P, alpha=1.0, w1=P, gate=None, rows=0, w2=P, eps=1e-6, so=P, y=V(8192), q=None, sc=None,
         r1=None, r2=None):
    return lib.moe_block_norm(ctypes.byref(s), x, r, alpha, w1, gate, rows, w2, eps, so, y, q, sc, r1, r2, None)


def test_block_norm_refusals(lib):
    assert _fwd(lib, NORM.replace(T=-1)) == EINVAL
    assert _fwd(lib, x=None) == EINVAL
    for name in ("x", "r", "w1", "w2", "so", "y"):
        assert _fwd(lib, **{name: V(4096 + 8)}) == EINVAL, name
    for bad in (float("nan"), float("inf")):
        assert _fwd(lib, alpha=bad) == EINVAL and _fwd(lib, eps=bad) == EINVAL
    assert _fwd(lib, eps=0.0) == EINVAL
    assert _fwd(lib, gate=P, rows=-1) == EINVAL
    assert _fwd(lib, gate=V(4097), rows=0) == EINVAL           # a bf16 value a token
    assert _fwd(lib, gate=V(4098), rows=1) == EINVAL           # rows of gates are vectors
    assert _fwd(lib, w1=None, r1=P) == EINVAL                  # no norm behind, no rstd of it
    for name in ("y", "q", "sc", "r2"):                        # no norm in front, nothing from it
        assert _fwd(lib, **{"w2": None, "y": None, name: P}) == EINVAL, name
    assert _fwd(lib, so=None, y=None) == EINVAL                # nothing to compute
    assert _fwd(lib, so=P, y=P) == EINVAL
    assert _fwd(lib, q=P) == EINVAL and _fwd(lib, sc=P) == EINVAL
    f = NORM.replace(H=68, dtype=moe.MOE_F32)
    assert _fwd(lib, f, q=P, sc=P) == EUNSUP
    assert _fwd(lib, NORM.replace(T=0), x=None, r=None, so=None, y=None) == 0


def _bwd(lib, s=NORM, x=P, r1=P, so=P, r2=P, alpha=1.0, w1=P, gate=None, rows=0, w2=P, dy=P, ds=P, dx=P, dr=V(8192),
         dw1=P, dg=None, dw2=P, ws=P, need=None):
    need = moe.moe_block_norm_backward_workspace_bytes(s, rows if gate else 0) if need is None else need
    return lib.moe_block_norm_backward(ctypes.byref(s), x, r1, so, r2, alpha, w1, gate, rows, w2, dy, ds, dx, dr, dw1, dg,
                                       dw2, ws, need, None)


def test_block_norm_backward_refusals(lib):
    f = moe.moe_block_norm_backward_workspace_bytes
    assert f(NORM) >= 2 * 16 * 64 * 4 and f(NORM, -1) == 0 and f(NORM.replace(R=3)) == 0
    assert f(NORM, 16) >= 3 * 16 * 64 * 4                      # the gate's parts too
    for name in ("x", "r1", "so", "r2", "w2", "dx", "ws"):
        assert _bwd(lib, **{name: None}) == EINVAL, name
    for name in ("x", "so", "w1", "w2", "dy", "ds", "dx", "dr", "dw1", "dw2", "ws"):
        assert _bwd(lib, **{name: V(4096 + 8)}) == EINVAL, name
    assert _bwd(lib, r1=V(4097)) == EINVAL and _bwd(lib, r2=V(4098)) == EINVAL
    assert _bwd(lib, alpha=float("nan")) == EINVAL
    assert _bwd(lib, dy=None, ds=None, dw2=None) == EINVAL     # no gradient comes in
    assert _bwd(lib, dy=None) == EINVAL                        # dw_pre without dy
    assert _bwd(lib, w1=None) == EINVAL                        # dw_post without w_post
    assert _bwd(lib, dg=P) == EINVAL                           # dgate without a gate
    assert _bwd(lib, gate=P, rows=-1) == EINVAL
    assert _bwd(lib, gate=P, rows=3, dg=V(4100)) == EINVAL
    assert _bwd(lib, dx=P, dr=P) == EINVAL
    assert _bwd(lib, need=moe.moe_block_norm_backward_workspace_bytes(NORM) - 1) == EINVAL
    assert _bwd(lib, gate=P, rows=16, need=moe.moe_block_norm_backward_workspace_bytes(NORM)) == EINVAL
    assert _bwd(lib, NORM.replace(T=0), dx=None, dr=None, dw1=None, dw2=None) == 0


@pytest.mark.parametrize("name", ["moe_mx4_quantize", "moe_mx4_dequantize"])
def test_mx4_refusals(lib, name):
    f = getattr(lib, name)
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


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    s = moe.Shape(4, 64, 8, 2, 128, 4, 2, moe.MOE_F32)
    x, u8 = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.moe_block_norm(s, x, 1e-6, s=x)
    with pytest.raises(ValueError):
        moe.moe_block_norm_backward(s, x, None, None, x, x, x)
    with pytest.raises(ValueError):
        moe.moe_mx4_quantize(x, u8, u8)
    with pytest.raises(ValueError):
        moe.moe_mx4_dequantize(u8, u8, x)


# ------------------------------------------------ the float64 forms themselves ----

def test_the_scale_and_codes_by_hand():
    torch = pytest.importorskip("torch")
    import step_ref as ref

    v = torch.zeros(4, 32, dtype=torch.float64)
    v[0, :9] = torch.tensor([6.0, 5.0, 2.5, 3.5, 0.25, 0.75, 1.25, -1.75, 5.0000001],
                            dtype=torch.float64)   # scale 1, ties to even codes
    v[1, 0], v[1, 1] = 6.0000001, 1.0                                                   # scale 2
    v[2, 3] = 2.0 ** -130                                                               # the smallest scale
    v[3, 5] = float("inf")
    c, s = ref.codes4(v)
    assert s[:, 0].tolist() == [127, 128, 0, 255]
    assert c[0, :9].tolist() == [7, 6, 4, 6, 0, 2, 2, 12, 7]
    assert c[1, :2].tolist() == [5, 1]
    assert c[2, 3] == 0 and c[3].sum() == 0       # 2^-130 is 1/8 of the scale
    assert ref.values4(ref.pack4(c), s)[0, :4].tolist() == [6.0, 4.0, 2.0, 4.0]


@pytest.mark.parametrize("gate_kind", ["none", "token", "channel", "groups", "values"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_the_backward_form_against_differences(gate_kind, post, pre):
    torch = pytest.importorskip("torch")
    import step_ref as ref

    T, H, eps, alpha, h = 5, 12, 1e-3, 0.75, 1e-6
    torch.manual_seed(3)
    p = {"x": torch.randn(T, H), "residual": torch.randn(T, H), "w_post": 1 + 0.3 * torch.randn(H),
         "w_pre": 1 + 0.3 * torch.randn(H)}
    rows = {"none": 0, "token": 0, "channel": T, "groups": 2, "values": 1}[gate_kind]
    if gate_kind != "none":
        p["gate"] = torch.randn(T) if rows == 0 else torch.randn(-(-T // rows), H)
    p = {n: v.double() for n, v in p.items() if (post or n != "w_post") and (pre or n != "w_pre")}
    dy, ds = torch.randn(T, H).double(), torch.randn(T, H).double()

    def forward(q):
        s, _, r1 = ref.block_norm(q["x"], q["residual"], alpha, q.get("w_post"), q.get("gate"), rows, None, eps)
        loss = (s * ds).sum()
        r2 = ref.rstd(s, eps)[:, 0]
        if pre:
            loss = loss + (s * r2[:, None] * q["w_pre"] * dy).sum()
        return loss, s, r1, r2

    _, s, r1, r2 = forward(p)
    got = ref.block_norm_bwd(p["x"], r1, s, r2, alpha, p.get("w_post"), p.get("gate"), rows, p.get("w_pre"),
                             dy if pre else None, ds)
    names = {"x": "dx", "residual": "dresidual", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
    assert set(got) == {names[n] for n in p}
    for n, v in p.items():
        num = torch.zeros_like(v).reshape(-1)
        for i in range(v.numel()):
            e = torch.zeros_like(v).reshape(-1)
            e[i] = h
            e = e.view(v.shape)
            num[i] = (forward({**p, n: v + e})[0] - forward({**p, n: v - e})[0]) / (2 * h)
        # differences of step h: h^2 of third derivatives, and 2^-52 / h of the loss
        assert torch.allclose(got[names[n]][0].reshape(-1), num, rtol=1e-6, atol=1e-7), n


# ------------------------------------------------------- the layer for a few tokens ----

def _few(lib, s, form=1, x=P, wr=P, bias=None, routed=(P,) * 6, shared=None, SF=0, out=P, ids=None, w=None, err=P, ws=P,
         need=None):
    from expert_load_balance_amd.step import FewWeightsT

    need = lib.moe_few_workspace_bytes(ctypes.byref(s), form, SF) if need is None else need
    a = None if routed is None else ctypes.byref(FewWeightsT(*routed))
    b = None if shared is None else ctypes.byref(FewWeightsT(*shared))
    return lib.moe_few_layer(ctypes.byref(s), form, x, wr, bias, a, b, SF, out, ids, w, err, ws, need, None)


def test_few_layer_refusals(lib):
    s = moe.Shape(4, 128, 8, 2, 128, 1, 0, moe.MOE_BF16)
    size = moe.moe_few_workspace_bytes
    assert size(s, moe.MOE_W_MX8) >= 4 * 8 * 4 + 2 * 8 * 128 * 2 + 8 * 128 * 4
    assert size(s, moe.MOE_W_MX4, 128) > size(s, moe.MOE_W_MX4)
    for bad, st in [(s.replace(T=33), EUNSUP), (s.replace(dtype=moe.MOE_F32), EUNSUP), (s.replace(H=192), EUNSUP),
                    (s.replace(F=192), EUNSUP), (s.replace(H=8320), EUNSUP), (s.replace(E=0), EINVAL),
                    (s.replace(k=9), EINVAL), (s.replace(T=-1), EINVAL)]:
        assert size(bad, moe.MOE_W_MX8) == 0
        assert _few(lib, bad, need=1 << 40) == st, bad
    assert size(s.replace(H=192, F=192), moe.MOE_W_BF16) > 0
    assert size(s, 3) == 0 and size(s, -1) == 0 and size(s, 1, -128) == 0 and size(s, 1, 64) == 0
    assert _few(lib, s, form=3, need=1 << 40) == EINVAL
    for name in ("x", "wr", "out", "err", "ws", "routed"):
        assert _few(lib, s, **{name: None}) == EINVAL, name
    for name in ("x", "wr", "out", "ws"):
        assert _few(lib, s, **{name: V(4096 + 8)}) == EINVAL, name
    for name in ("bias", "ids", "w", "err"):
        assert _few(lib, s, **{name: V(4097)}) == EINVAL, name
    for i in range(6):
        for p in (None, V(4104)):
            w = [P] * 6
            w[i] = p
            assert _few(lib, s, routed=w) == EINVAL, i
            assert _few(lib, s, shared=w, SF=128) == EINVAL, i
            if i < 3:                                          # (scales are not read in bf16)
                assert _few(lib, s, form=0, routed=w) == EINVAL, i
    assert _few(lib, s, shared=(P,) * 6, SF=0) == EINVAL       # a shared expert without a width
    assert _few(lib, s, SF=128) == EINVAL                      # and the other way round
    assert _few(lib, s, need=size(s, 1) - 1) == EINVAL
    assert _few(lib, s.replace(T=0), x=None, out=None) == 0


def test_few_layer_wrapper_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    from expert_load_balance_amd.layer import MoeLayerFew

    s = moe.Shape(2, 128, 8, 2, 128, 1, 0, moe.MOE_BF16)
    with pytest.raises(ValueError):
        MoeLayerFew(s.replace(T=40), "cpu", weights="mx4")
    L = MoeLayerFew(s, "cpu", weights="mx4")
    x, w = torch.zeros(2, 128, dtype=torch.bfloat16), (torch.zeros(8, 128, 64, dtype=torch.uint8),) * 2
    with pytest.raises(ValueError):
        L.forward(x, torch.zeros(8, 128, dtype=torch.bfloat16), None, w, w, w)


def test_grouped_gemm_mx4_refusals(lib):
    s = moe.Shape(16, 128, 8, 2, 128, 4, 2, moe.MOE_BF16)
    need = moe.moe_mx4_workspace_bytes(s)
    assert need >= 32 * 128 + 32 * 4
    assert moe.moe_mx4_workspace_bytes(s.replace(H=192)) == 0 and moe.moe_mx4_workspace_bytes(s.replace(R=3)) == 0
    g = lib.moe_grouped_gemm_mx4
    for i in range(11):
        a = [P] * 11
        a[i] = None
        assert g(ctypes.byref(s), *a, need, None) == EINVAL, i
        if i != 2:                                            # (the plan is int32: 4-byte aligned)
            a[i] = V(4096 + 8)
            assert g(ctypes.byref(s), *a, need, None) == EINVAL, i
    assert g(ctypes.byref(s), *[P] * 11, need - 1, None) == EINVAL
    assert g(ctypes.byref(s.replace(H=64)), *[P] * 11, need, None) == EUNSUP
    assert g(ctypes.byref(s.replace(dtype=moe.MOE_F32)), *[P] * 11, need, None) == EUNSUP
