"""GPU parity of the experts on 4-bit weights (moe_grouped_gemm_mx4 and
MoeLayerMx with weight_bits 4). Every e2m1 value is an e4m3 value, so the float64
form and the bounds of the 8-bit experts hold for the same values in 8-bit codes."""
import math

import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerMx  # noqa: E402

import step_ref  # noqa: E402
import block_ref  # noqa: E402
from test_gpu_block import BF, DEV, MX_CASES, choose, gen, quantized, randn, say  # noqa: E402

pytestmark = pytest.mark.gpu


def fours(v):
    q = torch.empty(*v.shape[:-1], v.shape[-1] // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(*v.shape[:-1], v.shape[-1] // 32, dtype=torch.uint8, device=DEV)
    moe.moe_mx4_quantize(v.contiguous(), q, s)
    return q, s


def as_eights(w):
    """The same values as e4m3 codes, with the same scales."""
    t = torch.tensor(step_ref.E2M1 + tuple(-v for v in step_ref.E2M1), device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    return t[step_ref.unpack4(w[0]).long()], w[1]


def weights4(g, E, F, H):
    return tuple(fours(randn(g, E, *s) / math.sqrt(s[1])) for s in ((F, H), (F, H), (H, F)))


def check(L, xq, xs, ids, wts):
    """Every row of y within the float64 experts' bound, which grows with K, and all
    of them by norm: bf16's rounding leaves 2^-8 / sqrt(12) times about 1.5 (0.0017),
    and up to 0.3 % of h's codes that are the neighbour's, 2^-3 of a value off at
    most, sqrt(0.003) / 8 / sqrt(12) times about 1.5 (0.003) on the largest tiles:
    0.0035 together."""
    assert int(L.err.item()) == 0
    a, wts = block_ref.values(xq, xs), tuple(as_eights(v) for v in wts)
    flat, tok = ids.reshape(-1).long(), torch.arange(ids.numel(), device=DEV) // ids.shape[1]
    y, tol = block_ref.experts(a[tok], xs.view(torch.uint8)[tok], flat, *wts)
    got = L.y[L.dest_row.reshape(-1).long()].double()
    bad = ~((got - y).abs() <= (y.abs() + tol) * block_ref.HALF[BF] + tol + 1e-30)      # (a NaN is bad)
    off = float((got - y).norm() / y.norm())
    print("bound / y", float(tol.norm() / y.norm()), "error / y", off, flush=True)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values of y"
    assert off <= 0.0035, off


def run(L, xq, xs, ids, w, wts):
    for buf in (L.y, L.out):
        buf.fill_(float("nan"))
    L.mx_ws.fill_(0xFF)
    out = L.experts(xq, xs, ids, w, *wts).clone()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("case", MX_CASES + [
    (40, 7168, 4, 1, 8192, 2, 0.2, None), (300, 4096, 3, 2, 14336, 3, 0.4, None), (6300, 4096, 3, 1, 512, 1, 0.0, None),
    (2000, 1024, 6, 2, 384, 3, 2.0, None), (1500, 128, 5, 2, 2048, 1, 2.0, None),
], ids=lambda c: "T{}H{}E{}k{}F{}R{}".format(*c[:6]))
def test_experts_mx4(case):
    T, H, E, k, F, R, skew, only = case
    say("experts_mx4", case)
    g = gen(T + H + E + 1)
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, R, 1, moe.MOE_BF16), DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H) * torch.exp(randn(g, H)))
    ids, w = choose(g, T, E, k, skew, only)
    wts = weights4(g, E, F, H)
    out = run(L, xq, xs, ids, w, wts)
    y = L.y.clone()
    check(L, xq, xs, ids, wts)
    L.mx_ws.fill_(0x7F)
    L.experts(xq, xs, ids, w, *wts)
    assert torch.equal(L.out, out) and torch.equal(L.y, y)       # whatever the workspace held


def test_scales_far_apart_and_a_nan_in_a_row():
    T, H, E, k, F = 96, 512, 3, 1, 640
    g = gen(4)
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 1, 0, moe.MOE_BF16), DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H) * torch.exp2(torch.randint(-20, 20, (H // 32, 1), generator=g, device=DEV).float()
                                                   ).expand(H // 32, 32).reshape(H))
    ids, w = choose(g, T, E, k, 0.0)
    wts = weights4(g, E, F, H)
    for q, s in wts:
        s += torch.randint(-12, 12, s.shape, generator=g, device=DEV).to(torch.uint8)
    run(L, xq, xs, ids, w, wts)
    check(L, xq, xs, ids, wts)
    want = L.out.clone()
    xs[5, 3] = 255
    run(L, xq, xs, ids, w, wts)
    assert bool(torch.isnan(L.out[5]).all())
    keep = [t for t in range(T) if t != 5]
    assert torch.equal(L.out[keep], want[keep])


def test_float4_tensors_and_refusals():
    T, H, E, k, F = 8, 256, 4, 2, 128
    g = gen(6)
    shape = moe.Shape(T, H, E, k, F, 2, 0, moe.MOE_BF16)
    L = MoeLayerMx(shape, DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H))
    ids, w = choose(g, T, E, k, 0.0)
    wts = weights4(g, E, F, H)
    out = run(L, xq, xs, ids, w, wts)
    if hasattr(torch, "float4_e2m1fn_x2"):
        typed = tuple((q.view(torch.float4_e2m1fn_x2), s.view(torch.float8_e8m0fnu)) for q, s in wts)
        assert torch.equal(run(L, xq, xs, ids, w, typed), out)
    with pytest.raises(ValueError):
        L.experts(xq, xs, ids, w, (wts[0][0][:3], wts[0][1]), *wts[1:])
    with pytest.raises(ValueError):
        MoeLayerMx(shape, DEV, weight_bits=6)


@pytest.mark.parametrize("H,F", [(640, 1152), (128, 384), (1152, 512)])
def test_a_nan_block_of_a_weight_stays_in_its_column(H, F):
    """The first block of a row of W_down, next to the end of the row before it."""
    T, E, k = 40, 2, 1
    g = gen(H + F)
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 1, 0, moe.MOE_BF16), DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H))
    ids, w = choose(g, T, E, k, 0.0)
    wts = weights4(g, E, F, H)
    run(L, xq, xs, ids, w, wts)
    check(L, xq, xs, ids, wts)
    want, on = L.out.clone(), ids[:, 0] == 0
    wts[2][1][0, 70, 0] = 255
    run(L, xq, xs, ids, w, wts)
    cols = [c for c in range(H) if c != 70]
    assert bool(torch.isnan(L.out[on][:, 70]).all())
    assert torch.equal(L.out[on][:, cols], want[on][:, cols]) and torch.equal(L.out[~on], want[~on])


@pytest.mark.parametrize("T", [3, 700])
def test_experts_mx4_from_a_graph_beside_eager_calls(T):
    H, E, k, F = 512, 8, 2, 512
    g = gen(T)
    shape = moe.Shape(T, H, E, k, F, 4, 0, moe.MOE_BF16)
    A, B = MoeLayerMx(shape, DEV, weight_bits=4), MoeLayerMx(shape, DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H))
    ids, w = choose(g, T, E, k, 0.3)
    wts = weights4(g, E, F, H)
    A.experts(xq, xs, ids, w, *wts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.experts(xq, xs, ids, w, *wts)
    for i in range(4):
        q, s = quantized(randn(g, T, H) * (i + 1))
        xq.copy_(q)
        xs.copy_(s)
        A.experts(xq, xs, ids, w, *wts)
        B.out.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(A.out, B.out), i


def test_bf16_layer_on_dequantised_weights_agrees():
    """moe_mx4_dequantize hands the bf16 layer the same weights: beside the 8-bit
    rows and activations, both compute one function."""
    T, H, E, k, F = 32, 512, 4, 2, 512
    g = gen(8)
    shape = moe.Shape(T, H, E, k, F, 1, 0, moe.MOE_BF16)
    wts = weights4(g, E, F, H)
    plain = []
    for q, s in wts:
        v = torch.empty(*q.shape[:-1], q.shape[-1] * 2, dtype=BF, device=DEV)
        moe.moe_mx4_dequantize(q, s, v)
        assert torch.equal(v.double(), step_ref.values4(q, s))
        plain.append(v)
    L = MoeLayerMx(shape, DEV, weight_bits=4)
    x = randn(g, T, H).to(BF)
    xq, xs = quantized(x)
    ids, w = choose(g, T, E, k, 0.0)
    run(L, xq, xs, ids, w, wts)
    xd = x.double()
    want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for t in range(T):
        for j in range(k):
            G, U, D = (p[int(ids[t, j])].double() for p in plain)
            h = (xd[t] @ G.t())
            want[t] += w[t, j].double() * ((h * torch.sigmoid(h) * (xd[t] @ U.t())) @ D.t())
    # two roundings to e4m3 (2^-4 of a value at most, 0.026 of the norm at random), and bf16's
    assert float((L.out.double() - want).norm() / want.norm()) < 0.07


@pytest.mark.parametrize("T", [20, 90, 400])
@pytest.mark.parametrize("F", [128, 256, 384, 512])
def test_a_nan_block_beside_short_rows(T, F):
    """Rows of one and two stages: the bytes behind a row's scales are other rows'."""
    H, E = 256, 2
    g = gen(H + F + T)
    L = MoeLayerMx(moe.Shape(T, H, E, 1, F, 1, 0, moe.MOE_BF16), DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H))
    ids, w = choose(g, T, E, 1, 0.0)
    wts = weights4(g, E, F, H)
    run(L, xq, xs, ids, w, wts)
    check(L, xq, xs, ids, wts)
    want, on = L.out.clone(), ids[:, 0] == 0
    wts[2][1][0, 70:73] = 255
    run(L, xq, xs, ids, w, wts)
    cols = [c for c in range(H) if not 70 <= c < 73]
    assert bool(torch.isnan(L.out[on][:, 70:73]).all())
    assert torch.equal(L.out[on][:, cols], want[on][:, cols]) and torch.equal(L.out[~on], want[~on])
