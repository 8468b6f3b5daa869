"""GPU parity of the operators around the layer (include/moe_block.h) against
plain float64 forms (block_ref.py): the residual-add norm and its backward,
8-bit blocks, the 8-bit experts, the global gradient norm and clipping."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerMx, alloc  # noqa: E402

import block_ref as ref  # noqa: E402
import synth  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print("[case]", *a, flush=True)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def norm_shape(T, H, t):
    return moe.Shape(T, H, 1, 1, 64, 1, 0, moe.MOE_BF16 if t == BF else moe.MOE_F32)


# ------------------------------------------------------------------- norm ----

NORM_CASES = [
    # T, H, type, residual, 8-bit output
    (1, 64, BF, False, True), (1, 4096, BF, True, True), (3, 192, BF, True, True),
    (7, 576, BF, True, False), (2, 2112, BF, False, True), (5, 7168, BF, True, True),
    (3, 16448, BF, True, True), (2, 32768, BF, True, True),
    (2, 32832, BF, True, True),          # wider than the registers hold
    (3, 40000 // 64 * 64, BF, False, False),
    (1, 4, F32, False, False), (9, 12, F32, True, False), (4, 2052, F32, True, False),
    (33, 160, F32, True, True), (2, 4128, F32, False, True), (2, 16388, F32, True, False),
    (2, 20000, F32, True, True), (1021, 96, F32, True, True),
]


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: f"T{c[0]}H{c[1]}{'bf16' if c[2] == BF else 'f32'}"
                                                           f"{'r' if c[3] else ''}{'q' if c[4] else ''}")
def test_rmsnorm(case):
    T, H, t, has_r, mx = case
    say("rmsnorm", case)
    g = gen(T * 31 + H)
    x = (randn(g, T, H) * torch.exp(randn(g, H))).to(t)
    r = (randn(g, T, H) * 3).to(t) if has_r else None
    w = (1 + 0.3 * randn(g, H)).to(t)
    if T > 2:
        x[1] = 0                                   # a row of zeros
        if has_r:
            r[1] = 0
        x[2] = x[2] * 1e-12
    s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    q = torch.empty(T, H, dtype=torch.uint8, device=DEV) if mx else None
    sc = torch.empty(T, H // 32, dtype=torch.uint8, device=DEV) if mx else None
    moe.moe_rmsnorm(norm_shape(T, H, t), x, w, EPS, residual=r, s=s, y=y, q=q, scales=sc, rstd=rstd)
    torch.cuda.synchronize()
    rs, rr, v = ref.norm(x, r, w, EPS)
    assert torch.equal(s, rs)
    rel = ref.norm_rel(H)
    assert bool(((rstd.double() - rr).abs() <= rel * rr).all())
    d = v.abs() * rel
    tol = (v.abs() + d) * ref.HALF[t] + d
    assert bool(((y.double() - v).abs() <= tol).all())
    if mx:
        ref.check_blocks(q, sc, v, d, "norm")


def test_rmsnorm_outputs_one_by_one_and_in_place():
    """Each output alone has the bits it has among the others; s and y may
    replace the inputs."""
    for T, H, t in [(5, 512, BF), (3, 33024, BF), (4, 256, F32), (2, 16416, F32)]:
        say("in place", T, H, t)
        g = gen(H)
        sh = norm_shape(T, H, t)
        x, r, w = randn(g, T, H).to(t), randn(g, T, H).to(t), randn(g, H).to(t)

        def out(**want):
            o = dict(s=torch.empty_like(x), y=torch.empty_like(x), rstd=torch.empty(T, device=DEV),
                     q=torch.empty(T, H, dtype=torch.uint8, device=DEV),
                     scales=torch.empty(T, H // 32, dtype=torch.uint8, device=DEV))
            return {n: o[n] for n in want} if want else o

        full = out()
        moe.moe_rmsnorm(sh, x, w, EPS, residual=r, **full)
        for names in (["s"], ["y"], ["q", "scales"], ["rstd"], ["s", "q", "scales"], ["y", "rstd"]):
            o = out(**dict.fromkeys(names))
            moe.moe_rmsnorm(sh, x, w, EPS, residual=r, **o)
            for n in names:
                assert torch.equal(o[n], full[n]), (names, n)
        a, b = x.clone(), r.clone()
        moe.moe_rmsnorm(sh, a, w, EPS, residual=b, s=b, y=a)
        assert torch.equal(b, full["s"]) and torch.equal(a, full["y"])
        a, b = x.clone(), r.clone()
        moe.moe_rmsnorm(sh, a, w, EPS, residual=b, s=a, y=b)
        assert torch.equal(a, full["s"]) and torch.equal(b, full["y"])
        a, b = x.clone(), r.clone()
        moe.moe_rmsnorm(sh, a, w, EPS, residual=b, y=b)
        assert torch.equal(b, full["y"]) and torch.equal(a, x)


def test_rmsnorm_more_rows_than_one_launch_takes():
    """2^26 + 3 rows of 64 threads each are more threads than a launch holds."""
    T, H = (1 << 26) + 3, 4
    x = torch.zeros(T, H, device=DEV)
    some = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, (1 << 25) + 7, T - 1], device=DEV)
    g = gen(4)
    x[some], w = randn(g, len(some), H), 1 + 0.1 * randn(g, H)
    y, rstd = torch.full_like(x, 9.0), torch.zeros(T, device=DEV)
    moe.moe_rmsnorm(norm_shape(T, H, F32), x, w, EPS, y=y, rstd=rstd)
    _, rr, v = ref.norm(x[some], None, w, EPS)
    assert bool(((y[some].double() - v).abs() <= v.abs() * (ref.norm_rel(H) + ref.HALF[F32])).all())
    assert bool(((rstd[some].double() - rr).abs() <= rr * ref.norm_rel(H)).all())
    assert int((y != 0).any(-1).sum()) == len(some) and bool((rstd > 0).all())


@pytest.mark.parametrize("t,H", [(BF, 4160), (BF, 576), (F32, 2080)], ids=["bf16", "bf16_narrow", "f32"])
def test_norms_past_the_caches(t, H):
    """Calls of more than 256 MB (their accesses are streamed) give the bits of
    the same rows in calls of 1000, in place as well."""
    T = 300_000_000 // (H * 4 * (2 if t == BF else 4)) + 7
    say("norms past the caches", T, H, t)
    g = gen(H)
    x, r, dy = (randn(g, T, H).to(t) for _ in range(3))
    w = (1 + 0.3 * randn(g, H)).to(t)

    def outs(n):
        return dict(s=torch.empty(n, H, dtype=t, device=DEV), y=torch.empty(n, H, dtype=t, device=DEV),
                    q=torch.empty(n, H, dtype=torch.uint8, device=DEV),
                    scales=torch.empty(n, H // 32, dtype=torch.uint8, device=DEV), rstd=torch.empty(n, device=DEV))

    big = outs(T)
    moe.moe_rmsnorm(norm_shape(T, H, t), x, w, EPS, residual=r, **big)
    dx, dw, dw1 = torch.empty_like(x), torch.empty(H, device=DEV), torch.empty(H, device=DEV)

    def back(n, s, rstd, dyn, ds, out, dwn):
        sh = norm_shape(n, H, t)
        ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(sh), dtype=torch.uint8, device=DEV)
        moe.moe_rmsnorm_backward(sh, s, w, rstd, dyn, out, dwn, ws, ds=ds)

    back(T, big["s"], big["rstd"], dy, r, dx, dw)
    total = torch.zeros(H, dtype=torch.float64, device=DEV)
    for i in range(0, T, 1000):
        n = min(1000, T - i)
        rows, o = slice(i, i + n), outs(n)
        moe.moe_rmsnorm(norm_shape(n, H, t), x[rows], w, EPS, residual=r[rows], **o)
        for name in o:
            assert torch.equal(big[name][rows], o[name]), (name, i)
        part = torch.empty(n, H, dtype=t, device=DEV)
        back(n, o["s"], o["rstd"], dy[rows], r[rows], part, dw1)
        assert torch.equal(dx[rows], part), i
        total += dw1.double()
    # each sum adds in float32: up to T / 512 rows in turn, then 512 partial sums in 16 + 16 steps
    mag = (dy.double() * big["s"].double() * big["rstd"].double()[:, None]).abs().sum(0)
    assert bool(((dw.double() - total).abs() <= 2 * (T / 512 + 64) * ref.U * mag).all())
    a, b, d = x.clone(), r.clone(), dy.clone()
    moe.moe_rmsnorm(norm_shape(T, H, t), a, w, EPS, residual=b, s=b, y=a)
    assert torch.equal(b, big["s"]) and torch.equal(a, big["y"])
    back(T, big["s"], big["rstd"], d, r, d, dw1)
    assert torch.equal(d, dx) and torch.equal(dw1, dw)


def test_rmsnorm_nonfinite_rows_stay_apart():
    T, H = 6, 256
    g = gen(5)
    x, w = randn(g, T, H).to(BF), (1 + 0.1 * randn(g, H)).to(BF)
    clean = x.clone()
    x[1, 7], x[3, 100], x[4, 255] = float("nan"), float("inf"), -float("inf")
    got = {}
    for name, v in (("clean", clean), ("bad", x)):
        y = torch.empty_like(v)
        q, sc = torch.empty(T, H, dtype=torch.uint8, device=DEV), torch.empty(T, 8, dtype=torch.uint8, device=DEV)
        moe.moe_rmsnorm(norm_shape(T, H, BF), v, w, EPS, y=y, q=q, scales=sc)
        got[name] = (y, q, sc)
    for a, b in zip(got["clean"], got["bad"]):
        for row in (0, 2, 5):
            assert torch.equal(a[row], b[row])
    y, q, sc = got["bad"]
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3, 100])) and bool(torch.isnan(y[4, 255]))
    # the block that holds the NaN: scale 255 and NaN codes
    assert int(sc[1, 0]) == 255 and int(sc[3, 3]) == 255
    assert bool((q[1].view(-1) & 0x7F == 0x7F).all())


BWD_CASES = [(1, 64, BF, False), (1, 4096, BF, True), (3, 192, BF, True), (700, 576, BF, True),
             (1030, 64, BF, False), (130, 7168, BF, True), (3, 32832, BF, True), (520, 33024, BF, True),
             (1, 4, F32, False), (333, 1540, F32, False), (9, 12, F32, True), (513, 260, F32, True),
             (3, 16388, F32, True)]


@pytest.mark.parametrize("case", BWD_CASES, ids=lambda c: f"T{c[0]}H{c[1]}{'bf16' if c[2] == BF else 'f32'}"
                                                          f"{'d' if c[3] else ''}")
def test_rmsnorm_backward(case):
    T, H, t, has_ds = case
    say("rmsnorm_backward", case)
    g = gen(T * 7 + H)
    sh = norm_shape(T, H, t)
    s, w = (randn(g, T, H) * torch.exp(0.5 * randn(g, H))).to(t), (1 + 0.3 * randn(g, H)).to(t)
    dy, ds = randn(g, T, H).to(t), randn(g, T, H).to(t) if has_ds else None
    rstd = torch.empty(T, device=DEV)
    moe.moe_rmsnorm(sh, s, w, EPS, rstd=rstd)
    dx, dw = torch.empty_like(s), torch.full((H,), 7.0, device=DEV)
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(sh), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)                                 # stale sums are NaN
    moe.moe_rmsnorm_backward(sh, s, w, rstd, dy, dx, dw, ws, ds=ds)
    torch.cuda.synchronize()
    rx, tol, rw, mag = ref.norm_bwd(s, w, rstd, dy, ds)
    assert bool(((dx.double() - rx).abs() <= (rx.abs() + tol) * ref.HALF[t] + tol).all())
    # rows of one workgroup in turn, then at most 32 + 16 partial sums
    chain = math.ceil(T / 512) + 2 + 32 + 16
    assert bool(((dw.double() - rw).abs() <= mag * chain * ref.U + 1e-30).all())
    # in place over dy, over ds; and the same bits again
    a, dw2 = dy.clone(), torch.empty_like(dw)
    moe.moe_rmsnorm_backward(sh, s, w, rstd, a, a, dw2, ws, ds=ds)
    assert torch.equal(a, dx) and torch.equal(dw2, dw)
    if has_ds:
        a = ds.clone()
        moe.moe_rmsnorm_backward(sh, s, w, rstd, dy, a, dw2, ws, ds=a)
        assert torch.equal(a, dx) and torch.equal(dw2, dw)


def test_rmsnorm_backward_against_differences():
    """<dx, d> and <dweight, e> against central differences of the float64
    forward along random directions. With f three times differentiable along
    the line, a central difference of step h is off by h^2 f''' / 6; halving
    h shows that term, and the bound is four times what is left of it plus
    the kernel's float32 rounding."""
    T, H = 6, 132
    g = gen(11)
    s, w, dy = randn(g, T, H), 1 + 0.3 * randn(g, H), randn(g, T, H)
    sh = norm_shape(T, H, F32)
    rstd, dx, dw = torch.empty(T, device=DEV), torch.empty_like(s), torch.empty(H, device=DEV)
    moe.moe_rmsnorm(sh, s, w, EPS, rstd=rstd)
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(sh), dtype=torch.uint8, device=DEV)
    moe.moe_rmsnorm_backward(sh, s, w, rstd, dy, dx, dw, ws)

    def f(a, b):
        return float((a * (a.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * b * dy.double()).sum())

    for k in range(4):
        d, e = randn(g, T, H).double(), randn(g, H).double()
        a, b = s.double(), w.double()
        for got, step in ((float((dx.double() * d).sum()), lambda h: (f(a + h * d, b) - f(a - h * d, b)) / (2 * h)),
                          (float((dw.double() * e).sum()), lambda h: (f(a, b + h * e) - f(a, b - h * e)) / (2 * h))):
            coarse, fine = step(1e-3), step(5e-4)
            rounding = 64 * ref.U * float((dx.double() * d).abs().sum() + (dw.double() * e).abs().sum())
            assert abs(got - fine) <= 4 * abs(coarse - fine) + rounding + 1e-9 * abs(got)


def test_norms_without_rows():
    for t in (BF, F32):
        sh = norm_shape(0, 64, t)
        x = alloc((0, 64), t, DEV)
        w, dw = torch.ones(64, dtype=t, device=DEV), torch.full((64,), 3.0, device=DEV)
        moe.moe_rmsnorm(sh, x, w, EPS, y=x)
        ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(sh), dtype=torch.uint8, device=DEV)
        moe.moe_rmsnorm_backward(sh, x, w, alloc((0,), F32, DEV), x, x, dw, ws)
        assert bool((dw == 0).all())               # a sum over no rows


# ------------------------------------------------------------ 8-bit blocks ----

@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 32), (5, 96), (257, 160), (2, 3, 64), (1, 1 << 16)])
def test_quantize_is_exact(shape, t):
    """The input is known exactly, so scale bytes and codes have one value."""
    g = gen(sum(shape))
    # scales from 2^-140 to 2^120: subnormal blocks and the largest included
    x = randn(g, *shape) * torch.exp2(torch.randint(-140, 120, (*shape[:-1], shape[-1] // 32), generator=g,
                                                    device=DEV).float()).repeat_interleave(32, -1)
    x = x.to(t)
    x[..., :32][..., 5] = 0
    if x.numel() > 64:
        x.view(-1, 32)[1] = 0                      # a block of zeros
    q, s = torch.empty(shape, dtype=torch.uint8, device=DEV), torch.empty((*shape[:-1], shape[-1] // 32),
                                                                          dtype=torch.uint8, device=DEV)
    moe.moe_mx_quantize(x, q, s)
    want, byte = ref.blocks(x.double())
    assert torch.equal(s.long(), byte)
    assert torch.equal(ref.values(q, s), want)


def test_quantize_borders_and_nonfinite():
    x = torch.zeros(8, 32, device=DEV)
    x[0, 3] = 448.0                                 # exactly the largest code
    x[1, 3] = float(np.nextafter(np.float32(448), np.float32(1e9)))
    x[2, 0], x[2, 1:9] = 256.0, torch.tensor([17.0, 18, 19, 20, 21, 22, 23, 25], device=DEV)   # ties
    x[3, 31] = float("inf")
    x[4, 0] = float("nan")
    x[5, 0] = 3.4e38
    x[6, 0] = 1e-45                                 # the smallest subnormal
    q = torch.empty(8, 32, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(8, 1, dtype=torch.float8_e8m0fnu, device=DEV)
    moe.moe_mx_quantize(x, q, s)
    b, want = s.view(torch.uint8).reshape(-1).tolist(), ref.blocks(x.double())
    assert b[0] == 127 and b[1] == 128 and b[3] == b[4] == 255 and b[6] == b[7] == 0
    assert b == want[1].reshape(-1).tolist()
    assert bool(torch.isnan(q[3].float()).all()) and bool(torch.isnan(q[4].float()).all())
    for i in (0, 1, 2, 5, 6, 7):
        assert torch.equal(ref.values(q[i], s[i]), want[0][i])


def test_quantize_large_offsets():
    """More than 2^32 bytes of input: a block at the far end has its own value."""
    rows, cols = (1 << 31) // 4096 + 3, 4096
    x = torch.zeros(rows, cols, dtype=BF, device=DEV)
    x[-1, -32:] = torch.arange(32, device=DEV).to(BF)
    q, s = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rows, cols // 32, dtype=torch.uint8, device=DEV)
    s.fill_(77)
    moe.moe_mx_quantize(x, q, s)
    want, byte = ref.blocks(x[-1:].double())
    assert torch.equal(s[-1:].long(), byte) and torch.equal(ref.values(q[-1:], s[-1:]), want)
    assert int(s[:-1].max()) == 0 and int(q[:-1].max()) == 0


# ----------------------------------------------------------- 8-bit experts ----

def quantized(v):
    q = torch.empty(v.shape, dtype=torch.uint8, device=DEV)
    s = torch.empty((*v.shape[:-1], v.shape[-1] // 32), dtype=torch.uint8, device=DEV)
    moe.moe_mx_quantize(v.contiguous(), q, s)
    return q, s


def weights(g, E, F, H):
    return (quantized(randn(g, E, F, H) / math.sqrt(H)), quantized(randn(g, E, F, H) / math.sqrt(H)),
            quantized(randn(g, E, H, F) / math.sqrt(F)))


def choose(g, T, E, k, skew, only=None):
    """ids, gate weights; `only`: the experts that tokens may take."""
    logits = randn(g, T, E) - skew * torch.log1p(torch.arange(E, device=DEV).float())
    if only is not None:
        mask = torch.full((E,), -1e30, device=DEV)
        mask[torch.tensor(only, device=DEV)] = 0
        logits = logits + mask
    top = torch.topk(logits, k, dim=-1)
    return top.indices.to(torch.int32), torch.softmax(top.values, -1)


def check_layer(L, xq, xs, ids, w, wts):
    """The layer's buffers against the float64 experts: every row of y, and
    the combine's sum."""
    T, k, H = L.shape.T, L.shape.k, L.shape.H
    assert int(L.err.item()) == 0
    a = ref.values(xq, xs)
    flat, tok = ids.reshape(-1).long(), torch.arange(T * k, device=DEV) // k
    y, tol = ref.experts(a[tok], xs.view(torch.uint8)[tok], flat, *wts)
    rows = L.dest_row.reshape(-1).long()
    assert torch.equal(torch.sort(rows).values, torch.arange(T * k, device=DEV))
    assert torch.equal(L.buf_q[rows], xq.view(torch.uint8)[tok]) and torch.equal(L.buf_s[rows], xs.view(torch.uint8)[tok])
    got = L.y[rows].double()
    bad = ~((got - y).abs() <= (y.abs() + tol) * ref.HALF[BF] + tol + 1e-30)      # (a NaN is bad)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values of y, worst {float(((got - y).abs() / (tol + y.abs() * 2.0 ** -8 + 1e-30)).max()):.3g}"
    # (the bound says something: beside the values it is small)
    print("bound / y", float(tol.norm() / y.norm()), "error / y", float((got - y).norm() / y.norm()), flush=True)
    assert float(tol.norm()) <= 0.25 * float(y.norm())


MX_CASES = [
    # T, H, E, k, F, R, skew, only
    (1, 128, 1, 1, 128, 1, 0.0, None), (1, 128, 8, 2, 128, 4, 0.0, None), (2, 256, 4, 4, 128, 2, 0.0, None),
    (16, 384, 8, 2, 256, 4, 0.5, None),          # half a weight tile in the down projection
    (33, 128, 6, 3, 640, 3, 0.0, None), (64, 512, 16, 4, 384, 8, 1.0, None),
    (129, 256, 5, 2, 256, 5, 0.3, [0, 3]),       # idle experts
    (300, 640, 3, 1, 128, 3, 0.0, None), (257, 128, 1, 1, 384, 1, 0.0, None),
    (400, 256, 40, 8, 128, 8, 0.6, None), (1000, 384, 7, 2, 256, 7, 2.0, None),
    (77, 1024, 256, 8, 128, 32, 0.2, None), (530, 128, 4, 2, 1152, 1, 0.0, [1, 2]),
    (5, 4096, 12, 4, 1536, 4, 0.0, None), (250, 2048, 12, 4, 768, 12, 0.1, None),
    # 256-row tiles (H and F from 512 up), K of 4 to 9 stages, tails of each size
    (300, 512, 1, 1, 640, 1, 0.0, None), (900, 640, 3, 2, 768, 3, 0.3, None), (1100, 896, 4, 1, 1152, 2, 0.1, None),
    (530, 768, 2, 2, 512, 2, 0.0, None), (2100, 1152, 6, 2, 896, 3, 0.5, [0, 2, 3, 5]), (256, 1280, 1, 1, 512, 1, 0.0, None),
    # tiles of every kind in one launch, K-parts in each
    (600, 1024, 24, 2, 1536, 8, 1.5, None),
]


@pytest.mark.parametrize("case", MX_CASES, ids=lambda c: "T{}H{}E{}k{}F{}R{}".format(*c[:6]))
def test_experts_mx(case):
    T, H, E, k, F, R, skew, only = case
    say("experts_mx", case)
    g = gen(T + H + E)
    shape = moe.Shape(T, H, E, k, F, R, 1, moe.MOE_BF16)
    L = MoeLayerMx(shape, DEV)
    xq, xs = quantized(randn(g, T, H) * torch.exp(randn(g, H)))
    ids, w = choose(g, T, E, k, skew, only)
    wts = weights(g, E, F, H)
    for buf in (L.y, L.out):
        buf.fill_(float("nan"))
    L.mx_ws.fill_(0xFF)
    out = L.experts(xq, xs, ids, w, *wts)
    torch.cuda.synchronize()
    check_layer(L, xq, xs, ids, w, wts)
    again, y = out.clone(), L.y.clone()
    L.mx_ws.fill_(0x7F)
    L.experts(xq, xs, ids, w, *wts)
    assert torch.equal(L.out, again) and torch.equal(L.y, y)       # whatever the workspace held


@pytest.mark.parametrize("case", [(4200, 2, 4096), (280, 40, 1024), (6300, 3, 4096), (6200, 9, 4096)],
                         ids=["256-row tiles", "32-row tiles", "last round in halves", "uneven halves"])
def test_experts_mx_rows_4_kb_apart(case):
    """Whole rounds of tiles on rows a multiple of 4 KB apart, whose K starts
    are staggered: every row is written, and a sample of them (each tile's ends
    and its middle) is the float64 experts'."""
    T, E, F = case
    H = 4096
    say("experts_mx", case)
    g = gen(T)
    L = MoeLayerMx(moe.Shape(T, H, E, 1, F, 2 - E % 2, 1, moe.MOE_BF16), DEV)
    xq, xs = quantized(randn(g, T, H))
    ids, w = choose(g, T, E, 1, 0.0)
    wts = weights(g, E, F, H)
    L.y.fill_(float("nan"))
    L.experts(xq, xs, ids, w, *wts)
    torch.cuda.synchronize()
    assert int(L.err.item()) == 0 and bool(torch.isfinite(L.y).all())
    row = L.dest_row.reshape(-1).long()
    tok = torch.sort(row).indices[torch.cat([torch.arange(i, T, 64, device=DEV) for i in (0, 31, 63)])]
    a = ref.values(xq[tok], xs[tok])
    y, tol = ref.experts(a, xs[tok], ids[tok, 0].long(), *wts)
    got = L.y[row[tok]].double()
    assert bool(((got - y).abs() <= (y.abs() + tol) * ref.HALF[BF] + tol + 1e-30).all())
    # the bound adds F magnitudes where y adds F values of either sign, so
    # beside y it grows with sqrt(F): check_layer's 0.25, which holds for F up
    # to 1536, is 0.25 sqrt(4096 / 1536) = 0.41 here
    assert float(tol.norm()) <= 0.25 * max(1.0, math.sqrt(F / 1536)) * float(y.norm())


def test_experts_mx_scales_far_apart():
    """Rows and weights whose block scales span 2^-30 .. 2^30, and zero rows."""
    T, H, E, k, F = 70, 256, 4, 2, 256
    g = gen(3)
    far = torch.exp2(torch.randint(-30, 30, (T, H // 32), generator=g, device=DEV).float()).repeat_interleave(32, -1)
    x = randn(g, T, H) * far
    x[5] = 0
    wts = weights(g, E, F, H)
    wts = (quantized(randn(g, E, F, H) * 1e-9), wts[1], wts[2])     # gate small: silu stays smooth
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 2, 1, moe.MOE_BF16), DEV)
    xq, xs = quantized(x)
    ids, w = choose(g, T, E, k, 0.0)
    L.experts(xq, xs, ids, w, *wts)
    torch.cuda.synchronize()
    check_layer(L, xq, xs, ids, w, wts)
    assert bool((L.y[L.dest_row[5].long()] == 0).all())


def test_experts_mx_nan_stays_in_its_row():
    T, H, E, k, F = 100, 128, 3, 1, 128
    g = gen(8)
    xq, xs = quantized(randn(g, T, H))
    ids, w = choose(g, T, E, k, 0.0)
    wts = weights(g, E, F, H)
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 1, 0, moe.MOE_BF16), DEV)
    clean = L.experts(xq, xs, ids, w, *wts).clone()
    xq[40, 17] = 0x7F                               # a NaN code
    xs[60, 1] = 255                                 # a NaN scale
    got = L.experts(xq, xs, ids, w, *wts)
    rest = [t for t in range(T) if t not in (40, 60)]
    assert torch.equal(got[rest], clean[rest])
    assert bool(torch.isnan(got[40]).all()) and bool(torch.isnan(got[60]).all())


def test_experts_mx_of_refused_ids():
    """Ids that the count flags: an expert named by every choice of a token
    (it then has more rows than there are tokens), and ids out of range, whose
    rows are left out of the sum."""
    T, H, E, k, F = 40, 1024, 4, 4, 1024
    g = gen(12)
    xq, xs = quantized(randn(g, T, H))
    wts = weights(g, E, F, H)
    _, w = choose(g, T, E, k, 0.0)
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 2, 1, moe.MOE_BF16), DEV)
    ids = torch.full((T, k), 2, dtype=torch.int32, device=DEV)
    L.y.fill_(float("nan"))
    L.experts(xq, xs, ids, w, *wts)
    torch.cuda.synchronize()
    assert int(L.err.item()) == moe.ERR_REPEAT
    L.err.zero_()
    check_layer(L, xq, xs, ids, w, wts)
    # out of range: the rest of the token's choices count
    ids, w = choose(g, T, E, k, 0.0)
    ids[:, 1], ids[7, 3] = -1, E
    check_kept(L, xq, xs, ids, w, wts)
    # so many rows that no tile would be cut along K, all but a few of them out
    # of range
    T = 49152
    xq, xs = quantized(randn(g, T, H))
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 2, 1, moe.MOE_BF16), DEV)
    ids, w = torch.full((T, k), -1, dtype=torch.int32, device=DEV), torch.rand(T, k, generator=g, device=DEV)
    ids[5:60, 0], ids[40000:40300, 2] = 1, 3
    check_kept(L, xq, xs, ids, w, wts)


def check_kept(L, xq, xs, ids, w, wts):
    """The layer's sum over the choices that are in range."""
    T, k, H, E = L.shape.T, L.shape.k, L.shape.H, L.shape.E
    L.y.fill_(float("nan"))
    out = L.experts(xq, xs, ids, w, *wts).double()
    torch.cuda.synchronize()
    assert int(L.err.item()) & moe.ERR_RANGE             # (and REPEAT where a token names one twice)
    flat, tok = ids.reshape(-1).long(), torch.arange(T * k, device=DEV) // k
    kept = (flat >= 0) & (flat < E)
    assert torch.equal(L.dest_row.reshape(-1) >= 0, kept)
    a = ref.values(xq, xs)[tok[kept]]
    y, tol = ref.experts(a, xs[tok[kept]], flat[kept], *wts)
    y, tol, ww = y, tol + y.abs() * ref.HALF[BF], w.reshape(-1)[kept].double()[:, None]
    want = torch.zeros(T, H, dtype=torch.float64, device=DEV).index_add_(0, tok[kept], y * ww)
    room = torch.zeros_like(want).index_add_(0, tok[kept], tol * ww + (y * ww).abs() * 8 * ref.U)
    assert bool(((out - want).abs() <= (want.abs() + room) * ref.HALF[BF] + room + 1e-30).all())


def test_experts_mx_without_tokens():
    L = MoeLayerMx(moe.Shape(0, 128, 4, 2, 128, 2, 1, moe.MOE_BF16), DEV)
    wts = weights(gen(1), 4, 128, 128)
    xq, xs = alloc((0, 128), torch.uint8, DEV), alloc((0, 4), torch.uint8, DEV)
    out = L.experts(xq, xs, alloc((0, 2), torch.int32, DEV), alloc((0, 2), F32, DEV), *wts)
    torch.cuda.synchronize()
    assert out.numel() == 0


def test_rows_behind_the_last_are_left():
    """Buffers longer than the shape needs keep what lies behind its rows."""
    T, H, E, k, F = 9, 256, 4, 2, 128
    g = gen(21)
    xq, xs = quantized(randn(g, T + 3, H))
    ids, w = choose(g, T, E, k, 0.0)
    wts = weights(g, E, F, H)
    L = MoeLayerMx(moe.Shape(T, H, E, k, F, 2, 1, moe.MOE_BF16), DEV)
    N = T * k
    L.buf_q = torch.full((N + 4, H), 9, dtype=torch.uint8, device=DEV)
    L.buf_s = torch.full((N + 4, H // 32), 9, dtype=torch.uint8, device=DEV)
    L.y = torch.full((N + 4, H), 9.0, dtype=BF, device=DEV)
    L.experts(xq, xs, ids, w, *wts)
    assert bool((L.y[N:] == 9).all()) and bool((L.buf_q[N:] == 9).all()) and bool((L.buf_s[N:] == 9).all())
    s = torch.full((T + 3, H), 9.0, dtype=BF, device=DEV)
    y, rstd = s.clone(), torch.full((T + 3,), 9.0, device=DEV)
    x, wn = randn(g, T, H).to(BF), torch.ones(H, dtype=BF, device=DEV)
    moe.moe_rmsnorm(norm_shape(T, H, BF), x, wn, EPS, s=s, y=y, rstd=rstd)
    assert bool((s[T:] == 9).all()) and bool((y[T:] == 9).all()) and bool((rstd[T:] == 9).all())


def test_rmsnorm_backward_of_a_very_wide_row():
    """2^28 + 64 columns: 16 threads a column are more than a launch holds."""
    H = (1 << 28) + 64
    s, w, dy = (torch.zeros(1, H, device=DEV) for _ in range(3))
    some = torch.tensor([0, 5, (1 << 27) - 1, 1 << 27, (1 << 28) - 1, 1 << 28, H - 1], device=DEV)
    g = gen(6)
    for v in (s, w, dy):
        v[0, some] = 1 + randn(g, len(some)).abs()
    rstd = torch.full((1,), 0.5, device=DEV)
    sh = norm_shape(1, H, F32)
    dw = torch.full((H,), 9.0, device=DEV)
    ws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(sh), dtype=torch.uint8, device=DEV)
    dx = torch.empty_like(s)
    moe.moe_rmsnorm_backward(sh, s, w, rstd, dy, dx, dw, ws)
    want = dy[0, some].double() * s[0, some].double() * 0.5
    assert bool(((dw[some].double() - want).abs() <= want * 4 * ref.U).all())
    assert int((dw != 0).sum()) == len(some) and int((dx != 0).sum()) == len(some)


# ------------------------------------------------------- gradient norm, clip ----

def grad_ws(grads):
    return torch.empty(moe.moe_grad_workspace_bytes(grads), dtype=torch.uint8, device=DEV)


def grad_norm(grads):
    norm, err = torch.full((1,), -1.0, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_grad_norm(grads, norm, err, grad_ws(grads))
    torch.cuda.synchronize()
    return norm, int(err.item())


def check_clip(grads, max_norm, in_place=False):
    norm, err = grad_norm(grads)
    want = math.sqrt(sum(float(g.double().pow(2).sum()) for g in grads))
    assert err == 0
    # fp64 sums, one rounding to float32
    assert abs(float(norm) - want) <= want * ref.U * 1.001
    into = [g.clone() for g in grads] if in_place else [torch.full_like(g, 5.0) for g in grads]
    src = into if in_place else grads
    moe.moe_grad_clip(src, into, max_norm, norm)
    torch.cuda.synchronize()
    if want > max_norm * (1 + 1e-6):
        c = max_norm / want
    elif want < max_norm * (1 - 1e-6):
        c = 1.0
    else:
        c = None
    for g, o in zip(grads, into):
        if c == 1.0:
            assert torch.equal(g, o)
        elif c is not None:
            r = g.double() * c
            # factor: the norm's and its own rounding; then the product's, then the type's
            # (below the smallest normal the half step is absolute)
            tol = r.abs() * (3.01 * ref.U + (ref.HALF[BF] if g.dtype == BF else 0)) + 2.0 ** -134
            assert bool(((o.double() - r).abs() <= tol).all())


GRAD_SETS = {
    "one": [((1,), F32)],
    "empty_among": [((0,), F32), ((7,), BF), ((0, 4), BF), ((3, 5), F32)],
    "odd": [((17,), BF), ((16385,), F32), ((16383,), BF), ((4, 4099), F32), ((33,), F32)],
    "many": [((i % 37 + 1,), F32 if i % 3 else BF) for i in range(400)],
    "chunks": [((3 << 20) + 5, F32), ((2 << 20) + 3, BF)],
    "batch_border": [((5 + i,), BF) for i in range(96)] + [((70000,), F32)],
}


@pytest.mark.parametrize("name", GRAD_SETS)
def test_grad_clip(name):
    say("grad_clip", name)
    g = gen(len(name))
    grads = [(randn(g, *(s if isinstance(s, tuple) else (s,))) * 10.0 ** (i % 5 - 3)).to(t)
             for i, (s, t) in enumerate(GRAD_SETS[name])]
    for max_norm in (1e-3, 1e9):
        check_clip(grads, max_norm)
        check_clip(grads, max_norm, in_place=True)


def test_grad_clip_views_at_odd_offsets():
    g = gen(4)
    base, low = randn(g, 40000), randn(g, 40000).to(BF)
    for off in (0, 1, 2, 3, 5):
        grads = [base[off:off + 16400 + off], low[off:off + 17000]]
        check_clip(grads, 0.5)
        norm, _ = grad_norm(grads)
        into = [torch.zeros(20001, device=DEV)[1:1 + grads[0].numel()], torch.zeros(20001, dtype=BF, device=DEV)[3:3 + 17000]]
        moe.moe_grad_clip(grads, into, 0.5, norm)
        c = 0.5 / float(norm)
        assert bool(((into[0].double() - grads[0].double() * c).abs() <= grads[0].double().abs() * c * 3.01 * ref.U + 1e-40).all())


def test_grad_clip_past_the_caches():
    """A list of more than 256 MB: its norm against float64, and the clip's bits
    against the same tensors' in lists of one."""
    g = gen(31)
    big = [randn(g, 40_000_003), randn(g, 30_000_001).to(BF), randn(g, 25_000_000)[1:], randn(g, 7).to(BF)]
    norm, err = grad_norm(big)
    want = math.sqrt(sum(float(t.double().pow(2).sum()) for t in big))
    assert err == 0 and abs(float(norm) - want) <= want * 2 * ref.U
    into = [torch.empty_like(t) for t in big]
    moe.moe_grad_clip(big, into, 1.0, norm)
    for t, o in zip(big, into):
        one = [torch.empty_like(t)]
        moe.moe_grad_clip([t], one, 1.0, norm)
        assert torch.equal(o, one[0])
    moe.moe_grad_clip(big, big, 1.0, norm)
    for t, o in zip(big, into):
        assert torch.equal(t, o)


def test_grad_norm_ranges_and_nonfinite():
    huge = torch.full((1000,), 1e30, device=DEV)              # squares pass float32
    tiny = torch.full((1 << 20,), 1e-30, device=DEV)          # squares vanish in float32
    n, e = grad_norm([huge])
    assert e == 0 and abs(float(n) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    n, e = grad_norm([tiny])
    assert e == 0 and abs(float(n) / (float(tiny[0]) * 1024) - 1) < 1e-6
    n, e = grad_norm([])
    assert e == 0 and float(n) == 0
    a = torch.ones(3, 3, device=DEV)
    n, e = grad_norm([a, a])                                  # listed twice: counted twice
    assert e == 0 and abs(float(n) - math.sqrt(18)) < 1e-6
    for bad in (float("nan"), float("inf")):
        v = torch.ones(50000, device=DEV)
        v[49999] = bad
        n, e = grad_norm([torch.ones(5, dtype=BF, device=DEV), v])
        assert e & moe.ERR_NONFINITE and not math.isfinite(float(n))
        into = [torch.zeros_like(v)]
        moe.moe_grad_clip([v], into, 1.0, n)                  # left as they are
        assert torch.equal(into[0].nan_to_num(3.0), v.nan_to_num(3.0))
    v = [torch.ones(10, device=DEV)]
    n, _ = grad_norm(v)
    moe.moe_grad_clip(v, v, 0.0, n)
    assert bool((v[0] == 0).all())


# --------------------------------------------------- together, streams, graphs --

def step_inputs(g, shape):
    T, H, E = shape.T, shape.H, shape.E
    return dict(x=randn(g, T, H).to(BF), residual=randn(g, T, H).to(BF))


def model(g, shape):
    H, E, F = shape.H, shape.E, shape.F
    return dict(norm_weight=(1 + 0.1 * randn(g, H)).to(BF), w_router=(randn(g, E, H) / math.sqrt(H)).to(BF),
                bias=None, wts=weights(g, E, F, H))


def run_step(L, inp, m, stream=None):
    return L.forward(inp["x"], inp["residual"], m["norm_weight"], EPS, m["w_router"], m["bias"], *m["wts"],
                     stream=stream)


@pytest.mark.parametrize("T", [1, 37, 200])
def test_serving_step(T):
    """Norm, router, 8-bit experts and combine as a model's step runs them."""
    shape = moe.Shape(T, 512, 16, 4, 384, 8, 1, moe.MOE_BF16)
    g = gen(T)
    m, inp, L = model(g, shape), step_inputs(g, shape), MoeLayerMx(shape, DEV)
    out, s = run_step(L, inp, m)
    torch.cuda.synchronize()
    rs, rr, v = ref.norm(inp["x"], inp["residual"], m["norm_weight"], EPS)
    assert torch.equal(s, rs)
    ref.check_blocks(L.xq, L.xs, v, v.abs() * ref.norm_rel(512), "step")
    check_layer(L, L.xq, L.xs, L.ids, L.w, m["wts"])
    # the combine's sum over y's rows, in float64
    y = L.y[L.dest_row.long()].double() * L.w.double()[..., None]
    tol = y.abs().sum(1) * 8 * ref.U
    assert bool(((out.double() - y.sum(1)).abs() <= (y.sum(1).abs() + tol) * ref.HALF[BF] + tol + 1e-30).all())
    # close to the same step on weights that were never rounded? the 8-bit
    # rows are within 2^-4 of the norm's, so the step is no more than noisy
    assert bool(torch.isfinite(out).all())


def test_serving_step_on_streams_and_in_a_graph():
    """A captured step replayed on new inputs, with eager work of the same
    objects between the replays, and two steps at once on two streams: the
    bits of the eager step."""
    shape = moe.Shape(48, 512, 16, 4, 384, 8, 1, moe.MOE_BF16)
    g = gen(77)
    m = model(g, shape)
    inputs = [step_inputs(g, shape) for _ in range(4)]
    L = MoeLayerMx(shape, DEV)
    want = []
    for inp in inputs:
        out, s = run_step(L, inp, m)
        want.append((out.clone(), s.clone()))
    # two streams, an object each
    A, B = torch.cuda.Stream(), torch.cuda.Stream()
    LA, LB = MoeLayerMx(shape, DEV), MoeLayerMx(shape, DEV)
    torch.cuda.synchronize()
    got = []
    for L2, st, inp in ((LA, A, inputs[0]), (LB, B, inputs[1]), (LA, A, inputs[2]), (LB, B, inputs[3])):
        out, s = run_step(L2, inp, m, stream=st)
        with torch.cuda.stream(st):
            got.append((out.clone(), s.clone()))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a graph
    G, static = MoeLayerMx(shape, DEV), {n: v.clone() for n, v in inputs[0].items()}
    run_step(G, static, m)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, s = run_step(G, static, m)
    for i in (1, 3, 0, 2, 1):
        for n in static:
            static[n].copy_(inputs[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(s, want[i][1]), i
        e, _ = run_step(L, inputs[(i + 1) % 4], m)          # eager work between
        assert torch.equal(e, want[(i + 1) % 4][0])


def test_training_step_norm_layer_clip():
    """Norm, the layer's forward and backward, the norm's backward and the
    clip of every gradient, chained as a step runs them (float32), against
    differences of a float64 forward of the same step with its choice of
    experts held; and the norm's backward and the clip replayed from a graph."""
    from expert_load_balance_amd.layer import MoeLayerBuffers

    T, H, E, k, F = 24, 64, 4, 2, 96
    shape = moe.Shape(T, H, E, k, F, 2, 1, moe.MOE_F32)
    g = gen(9)
    x, r, wn = randn(g, T, H), randn(g, T, H), 1 + 0.2 * randn(g, H)
    wr = randn(g, E, H) / 8
    wg, wu, wd = (randn(g, *s) / 8 for s in ((E, F, H), (E, F, H), (E, H, F)))
    L = MoeLayerBuffers(shape, DEV)
    s, xn, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    moe.moe_rmsnorm(shape, x, wn, EPS, residual=r, s=s, y=xn, rstd=rstd)
    logits = xn @ wr.t()
    out = L.forward(logits, None, xn, wg, wu, wd)
    # loss = <out + s, c>
    c = randn(g, T, H)
    N = T * k
    dy, dw = torch.empty(N, H, device=DEV), torch.empty(T, k, device=DEV)
    dbuf, dxn = torch.empty(N, H, device=DEV), torch.empty(T, H, device=DEV)
    gg, gu, gd = torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(wd)
    bws = torch.empty(moe.moe_backward_workspace_bytes(shape), dtype=torch.uint8, device=DEV)
    dlog = torch.empty(T, E, device=DEV)
    moe.moe_combine_backward(shape, c, L.y, L.dest_row, L.w, dy, dw)
    moe.moe_ffn_backward(shape, L.buf, L.plan, wg, wu, wd, dy, dbuf, gg, gu, gd, bws)
    moe.moe_permute_backward(shape, dbuf, L.dest_row, dxn)
    moe.moe_route_backward(shape, L.ids, L.w, dw, dlog)
    dxn += dlog @ wr
    gr = dlog.t() @ xn
    dx, gn = torch.empty_like(x), torch.empty(H, device=DEV)
    nws = torch.empty(moe.moe_rmsnorm_backward_workspace_bytes(shape), dtype=torch.uint8, device=DEV)
    moe.moe_rmsnorm_backward(shape, s, wn, rstd, dxn, dx, gn, nws, ds=c)
    grads = [gn, gr, gg, gu, gd]
    torch.cuda.synchronize()

    ids = L.ids.long()

    def loss(x, wn, wr, wg, wu, wd):
        s = x + r.double()
        xn = s * (s.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() * wn
        w = torch.softmax(torch.gather(xn @ wr.t(), 1, ids), -1)
        o = s
        for j in range(k):
            G, U, D = wg[ids[:, j]], wu[ids[:, j]], wd[ids[:, j]]
            a, b = torch.matmul(G, xn[..., None])[..., 0], torch.matmul(U, xn[..., None])[..., 0]
            o = o + w[:, j:j + 1] * torch.matmul(D, (a * torch.sigmoid(a) * b)[..., None])[..., 0]
        return float((o * c.double()).sum())

    at = [t.double() for t in (x, wn, wr, wg, wu, wd)]
    for i, got in enumerate([dx] + grads):
        d = randn(g, *at[i].shape).double()

        def step(h):
            p, m = list(at), list(at)
            p[i], m[i] = at[i] + h * d, at[i] - h * d
            return (loss(*p) - loss(*m)) / (2 * h)

        coarse, fine = step(1e-4), step(5e-5)
        mine = float((got.double() * d).sum())
        # float32 sums of up to max(T, F, H) terms on the way to each element
        tol = 4 * abs(coarse - fine) + 512 * ref.U * float((got.double() * d).abs().sum()) + 1e-6 * abs(mine)
        assert abs(mine - fine) <= tol, (i, mine, fine, tol)
    for m in (0.1, 1e6):
        check_clip(grads, m)
        check_clip(grads, m, in_place=True)
    # the same tail of the step from a graph, several times
    norm, err, ws = torch.empty(1, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), grad_ws(grads)
    into = [torch.empty_like(t) for t in grads]

    def tail():
        moe.moe_rmsnorm_backward(shape, s, wn, rstd, dxn, dx, gn, nws, ds=c)
        moe.moe_grad_norm(grads, norm, err, ws)
        moe.moe_grad_clip(grads, into, 0.1, norm)

    tail()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tail()
    for i in range(4):
        gg.mul_(1.5)
        dxn.mul_(0.9)
        tail()
        torch.cuda.synchronize()
        want = [norm.clone(), dx.clone()] + [t.clone() for t in into]
        for t in (norm, dx, *into):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, [norm, dx] + into):
            assert torch.equal(a, b), i
    assert int(err.item()) == 0
