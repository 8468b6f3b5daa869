"""GPU parity of the operators of include/moe_step.h against plain float64 forms
(step_ref.py): the norms between two blocks and their backward, 4-bit blocks."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402

import block_ref  # noqa: E402
import step_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 2.0 ** -20
ALPHA = 0.875
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print("[case]", *a, flush=True)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def shape_of(T, H, t):
    return moe.Shape(T, H, 1, 1, 64, 1, 0, moe.MOE_BF16 if t == BF else moe.MOE_F32)


def guarded(n, dtype):
    """n elements with a marked tail behind them, and a check of the tail."""
    full = torch.full((n + 64,), 113, dtype=torch.uint8, device=DEV) if dtype == torch.uint8 else \
        torch.full((n + 64,), 113.0, dtype=dtype, device=DEV)
    return full[:n], lambda: bool((full[n:] == 113).all())


# ------------------------------------------------------ norms between two blocks ----

# T, H, type, rows of the gate (None: no gate, 0: a value a token), residual, w_post, w_pre
CASES = [
    (1, 64, BF, None, True, True, True), (1, 4096, BF, 1, True, True, True), (3, 192, BF, 0, True, True, True),
    (7, 576, BF, 3, True, True, True), (5, 7168, BF, 5, True, True, True), (6, 2112, BF, 100, False, True, True),
    (4, 512, BF, 2, True, False, True), (4, 512, BF, 0, True, True, False), (9, 640, BF, 1, False, False, False),
    (2, 12288, BF, 2, True, True, True), (3, 32768, BF, 0, True, True, True),
    (3, 32832, BF, 2, True, True, True), (3, 40000 // 64 * 64, BF, 0, True, True, True),   # wider than the registers hold
    (1, 4, F32, 1, True, True, True), (9, 12, F32, 4, True, True, True), (4, 2052, F32, 0, True, True, True),
    (33, 160, F32, None, True, True, True), (2, 16388, F32, 1, True, True, True), (3, 20000, F32, 2, False, True, True),
    (777, 96, F32, 37, True, True, True), (1500, 64, BF, 1, True, True, True), (1031, 128, BF, 1031, True, True, True),
    (1031, 128, BF, 0, True, True, True), (600, 64, F32, 2, True, False, True),
]


def ident(c):
    T, H, t, rows, r, w1, w2 = c
    return f"T{T}H{H}{'bf16' if t == BF else 'f32'}g{rows}{'r' if r else ''}{'p' if w1 else ''}{'n' if w2 else ''}"


def inputs(c, seed=0):
    T, H, t, rows, has_r, post, pre = c
    g = gen(T * 31 + H + seed)
    x = (randn(g, T, H) * torch.exp(randn(g, H))).to(t)
    r = (randn(g, T, H) * 3).to(t) if has_r else None
    if T > 2:
        x[1] = 0                                   # a row of zeros
        if has_r:
            r[1] = 0
        x[2] = x[2] * 1e-12
    w1 = (1 + 0.3 * randn(g, H)).to(t) if post else None
    w2 = (1 + 0.3 * randn(g, H)).to(t) if pre else None
    gate = None if rows is None else (randn(g, T) if rows == 0 else randn(g, -(-T // rows), H)).to(t)
    return x, r, w1, gate, rows or 0, w2


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_block_norm(case):
    T, H, t = case[:3]
    say("block_norm", case)
    x, r, w1, gate, rows, w2 = inputs(case)
    (s, s_ok), (y, y_ok) = guarded(T * H, t), guarded(T * H, t)
    (r1, r1_ok), (r2, r2_ok) = guarded(T, F32), guarded(T, F32)
    mx = w2 is not None and H % 32 == 0
    (q, q_ok), (sc, sc_ok) = guarded(T * H, torch.uint8), guarded(T * H // 32, torch.uint8)
    moe.moe_block_norm(shape_of(T, H, t), x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2,
                       s=s, y=y if w2 is not None else None, q=q if mx else None, scales=sc if mx else None,
                       rstd_post=r1 if w1 is not None else None, rstd_pre=r2 if w2 is not None else None)
    torch.cuda.synchronize()
    assert s_ok() and y_ok() and r1_ok() and r2_ok() and q_ok() and sc_ok()
    want, tol, want_r1 = ref.block_norm(x, r, ALPHA, w1, gate, rows, w2, EPS)
    s = s.view(T, H)
    ref.check(s, (want, tol), "s", t)
    if w1 is not None:
        ref.check(r1, (want_r1, 2 * ref.U * want_r1), "rstd_post")
    if w2 is None:
        return
    v, d, want_r2 = ref.pre_norm(s, w2, EPS)
    ref.check(r2, (want_r2, 2 * ref.U * want_r2), "rstd_pre")
    ref.check(y.view(T, H), (v, d), "y", t)
    if mx:
        block_ref.check_blocks(q.view(T, H), sc.view(T, H // 32), v, d + v.abs() * 1e-12, "q")


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_block_norm_backward(case):
    T, H, t = case[:3]
    say("block_norm_backward", case)
    x, r, w1, gate, rows, w2 = inputs(case)
    g = gen(T + H)
    shape = shape_of(T, H, t)
    s, r1, r2 = torch.empty_like(x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    moe.moe_block_norm(shape, x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2, s=s,
                       rstd_post=r1 if w1 is not None else None, rstd_pre=r2 if w2 is not None else None)
    dy = randn(g, T, H).to(t) if w2 is not None else None
    ds = randn(g, T, H).to(t) if w2 is None or T % 2 else None
    (dx, dx_ok), (dr, dr_ok) = guarded(T * H, t), guarded(T * H, t)
    (dw1, a_ok), (dw2, b_ok) = guarded(H, F32), guarded(H, F32)
    (dg, g_ok) = guarded(gate.numel(), F32) if gate is not None else (None, lambda: True)
    ws, ws_ok = guarded(moe.moe_block_norm_backward_workspace_bytes(shape, rows), torch.uint8)

    def call(**other):
        a = dict(dy=dy, ds=ds, dx=dx, dresidual=dr)
        a.update(other)
        moe.moe_block_norm_backward(shape, x, r1 if w1 is not None else None, a["dy"], a["ds"], a["dx"], ws, s=s,
                                    rstd_pre=r2, alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2,
                                    dresidual=a["dresidual"], dw_post=dw1 if w1 is not None else None, dgate=dg,
                                    dw_pre=dw2 if w2 is not None else None)

    call()
    torch.cuda.synchronize()
    assert dx_ok() and dr_ok() and a_ok() and b_ok() and g_ok() and ws_ok()
    want = ref.block_norm_bwd(x, r1, s, r2, ALPHA, w1, gate, rows, w2, dy, ds)
    got = {"dx": dx.view(T, H), "dresidual": dr.view(T, H), "dw_post": dw1, "dw_pre": dw2,
           "dgate": dg if dg is None else dg.view(gate.shape)}
    for name, bound in want.items():
        ref.check(got[name], bound, name, t if name in ("dx", "dresidual") else None)
    # again in place: dx over dy (or ds), the same bits
    keep = {n: v.clone() for n, v in got.items() if n in want}
    into = (dy if dy is not None else ds)
    call(dx=into, dresidual=ds if ds is not None and ds is not into else dr)
    torch.cuda.synchronize()
    assert torch.equal(into, keep["dx"])
    assert torch.equal(ds if ds is not None and ds is not into else dr.view(T, H), keep["dresidual"])
    for n in ("dw_post", "dw_pre", "dgate"):
        if n in want:
            assert torch.equal(got[n], keep[n]), n


@pytest.mark.parametrize("case", [(6, 256, F32, 4, True, True, True), (5, 128, F32, 0, True, True, True)], ids=ident)
def test_block_norm_backward_against_differences(case):
    """A directional derivative of the float64 forward, in every input at once."""
    T, H, t = case[:3]
    x, r, w1, gate, rows, w2 = inputs(case)
    x[1], r[1], x[2] = x[0] * 0.5, r[0] + 1, x[3] + 0.25      # (rows of zeros have no smooth neighbourhood of step h)
    g = gen(5)
    shape = shape_of(T, H, t)
    s, r1, r2 = torch.empty_like(x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    moe.moe_block_norm(shape, x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2, s=s,
                       rstd_post=r1, rstd_pre=r2)
    dy, ds = randn(g, T, H), randn(g, T, H)
    out = {n: torch.empty_like(v) for n, v in (("x", x), ("residual", r), ("w_post", w1), ("w_pre", w2), ("gate", gate))}
    ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(shape, rows), dtype=torch.uint8, device=DEV)
    moe.moe_block_norm_backward(shape, x, r1, dy, ds, out["x"], ws, s=s, rstd_pre=r2, alpha=ALPHA, w_post=w1, gate=gate,
                                gate_rows=rows, w_pre=w2, dresidual=out["residual"], dw_post=out["w_post"],
                                dgate=out["gate"], dw_pre=out["w_pre"])
    p = {"x": x.double(), "residual": r.double(), "w_post": w1.double(), "w_pre": w2.double(), "gate": gate.double()}

    def loss(q):
        z, _, _ = ref.block_norm(q["x"], q["residual"], ALPHA, q["w_post"], q["gate"], rows, None, EPS)
        return float((z * ds.double()).sum() + (z * ref.rstd(z, EPS) * q["w_pre"] * dy.double()).sum())

    h = 1e-6
    for n, v in p.items():
        u = torch.randn(v.shape, generator=g, device=DEV, dtype=torch.float64)
        num = (loss({**p, n: v + h * u}) - loss({**p, n: v - h * u})) / (2 * h)
        got, size = float((out[n].double() * u).sum()), float((out[n].double() * u).abs().sum())
        # float32 gradients of a few hundred roundings each, beside the differences' own 1e-7
        assert abs(got - num) <= 1e-4 * size, (n, got, num, size)


def test_block_norm_keeps_a_bad_row_to_itself():
    T, H = 5, 256
    x, r, w1, gate, rows, w2 = inputs((T, H, BF, 2, True, True, True), 7)
    shape = shape_of(T, H, BF)

    def run():
        s, y = torch.empty_like(x), torch.empty_like(x)
        moe.moe_block_norm(shape, x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2, s=s, y=y)
        torch.cuda.synchronize()
        return s, y

    s0, y0 = run()
    x[3, 7], r[4, 1] = float("nan"), float("inf")
    s1, y1 = run()
    assert torch.equal(s0[:3], s1[:3]) and torch.equal(y0[:3], y1[:3])
    assert bool(torch.isnan(s1[3]).all()) and bool(torch.isnan(y1[3]).all()) and bool(torch.isinf(s1[4, 1]))


def test_block_norm_in_place_and_no_rows():
    T, H = 6, 320
    x, r, w1, gate, rows, w2 = inputs((T, H, BF, 0, True, True, True), 9)
    shape = shape_of(T, H, BF)
    s, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_block_norm(shape, x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, w_pre=w2, s=s, y=y)
    moe.moe_block_norm(shape, x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, w_pre=w2, s=r, y=x)
    torch.cuda.synchronize()
    assert torch.equal(s, r) and torch.equal(y, x)
    none = moe.Shape(0, H, 1, 1, 64, 1, 0, moe.MOE_BF16)
    dw = torch.full((2, H), 5.0, device=DEV)
    ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(none, 0), dtype=torch.uint8, device=DEV)
    e, f = x[:0], torch.empty(0, device=DEV)
    moe.moe_block_norm_backward(none, e, f, e, e, e, ws, s=e, rstd_pre=f, w_post=w1, w_pre=w2, dw_post=dw[0], dw_pre=dw[1])
    torch.cuda.synchronize()
    assert not bool(dw.any())


@pytest.mark.parametrize("rows", [0, 3, 64])
def test_block_norm_step_from_a_graph_and_another_stream(rows):
    """Forward and backward captured, replayed beside eager calls of their own buffers."""
    T, H = 64, 1024
    case = (T, H, BF, rows, True, True, True)
    x, r, w1, gate, rows, w2 = inputs(case, 3)
    shape, g = shape_of(T, H, BF), gen(3)
    dy, ds = randn(g, T, H).to(BF), randn(g, T, H).to(BF)
    nws = moe.moe_block_norm_backward_workspace_bytes(shape, rows)

    def bufs():
        o = {n: torch.empty_like(x) for n in ("s", "y", "dx", "dr")}
        o.update(r1=torch.empty(T, device=DEV), r2=torch.empty(T, device=DEV), dw1=torch.empty(H, device=DEV),
                 dw2=torch.empty(H, device=DEV), dg=torch.empty(gate.shape, device=DEV),
                 ws=torch.empty(nws, dtype=torch.uint8, device=DEV))
        return o

    def step(o):
        moe.moe_block_norm(shape, x, EPS, residual=r, alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2, s=o["s"],
                           y=o["y"], rstd_post=o["r1"], rstd_pre=o["r2"])
        moe.moe_block_norm_backward(shape, x, o["r1"], dy, ds, o["dx"], o["ws"], s=o["s"], rstd_pre=o["r2"], alpha=ALPHA,
                                    w_post=w1, gate=gate, gate_rows=rows, w_pre=w2, dresidual=o["dr"], dw_post=o["dw1"],
                                    dgate=o["dg"], dw_pre=o["dw2"])

    a, b, c = bufs(), bufs(), bufs()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    side = torch.cuda.Stream()
    for i in range(4):
        x.mul_(1.25)
        dy.mul_(-0.5)
        torch.cuda.synchronize()
        step(a)
        with torch.cuda.stream(side):
            step(c)
        graph.replay()
        torch.cuda.synchronize()
        for n in a:
            if n != "ws":
                assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n]), (i, n)


# ---------------------------------------------------------------- 4-bit blocks ----

def quantize(x):
    q = torch.empty(*x.shape[:-1], x.shape[-1] // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(*x.shape[:-1], x.shape[-1] // 32, dtype=torch.uint8, device=DEV)
    moe.moe_mx4_quantize(x, q, s)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (129, 2080), (7, 4096), (2, 64 * 1024 + 32), (4099, 64)])
def test_mx4_quantize(rows, cols, t):
    say("mx4", rows, cols, t)
    g = gen(rows + cols)
    x = randn(g, rows, cols) * torch.exp2(torch.randint(-40, 40, (rows, cols // 32, 1), generator=g, device=DEV).float()
                                          ).expand(rows, cols // 32, 32).reshape(rows, cols)
    x = x.to(t)
    q, s = quantize(x)
    codes, want = ref.codes4(x.double())
    assert torch.equal(s, want) and torch.equal(q, ref.pack4(codes))
    for o in (BF, F32):
        v = torch.empty(rows, cols, dtype=o, device=DEV)
        moe.moe_mx4_dequantize(q, s, v)
        torch.cuda.synchronize()
        assert torch.equal(v, ref.values4(q, s).to(o))


def test_mx4_borders():
    """Every midpoint and its neighbours, every scale's border, both types."""
    for t in (BF, F32):
        step = torch.finfo(t).eps
        for e in (-126, -60, -1, 0, 1, 60, 120):
            edge = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0], dtype=torch.float64)
            v = torch.cat([edge, edge * (1 + step), edge * (1 - step / 2)])
            v = v[v <= 6]
            v = torch.cat([v, -v])
            rows = torch.zeros(len(v), 32, dtype=torch.float64)
            rows[:, 0], rows[:, 1] = 6.0, v
            rows2 = torch.zeros(len(v), 32, dtype=torch.float64)
            rows2[:, 31] = v                         # and as the block's largest
            x = (torch.cat([rows, rows2]) * 2.0 ** e).to(t).to(DEV)
            q, s = quantize(x)
            codes, want = ref.codes4(x.double())
            assert torch.equal(s, want), (t, e)
            assert torch.equal(q, ref.pack4(codes)), (t, e)


def test_mx4_special_values():
    for t in (BF, F32):
        x = torch.randn(8, 64, device=DEV).to(t)
        x[0, 3], x[1, 40], x[2, 63] = float("inf"), float("nan"), -float("inf")
        x[3] = 0
        x[4] = torch.finfo(t).max
        x[5] = torch.finfo(t).smallest_normal
        x[6] = -0.0
        q, s = quantize(x)
        codes, want = ref.codes4(x.double())
        assert torch.equal(s, want) and torch.equal(q, ref.pack4(codes))
        v = torch.empty_like(x)
        moe.moe_mx4_dequantize(q, s, v)
        torch.cuda.synchronize()
        w = ref.values4(q, s).to(t)
        assert torch.equal(torch.isnan(v), torch.isnan(w)) and torch.equal(v[~torch.isnan(w)], w[~torch.isnan(w)])
        assert bool(torch.isnan(v[0, :32]).all()) and not bool(torch.isnan(v[0, 32:]).any())


def test_mx4_every_code_and_scale():
    byte = torch.arange(256, device=DEV).to(torch.uint8)
    q = (torch.arange(16, device=DEV).to(torch.uint8) * 17).expand(256, 16).contiguous()
    s = byte[:, None].contiguous()
    for t in (BF, F32):
        v = torch.empty(256, 32, dtype=t, device=DEV)
        moe.moe_mx4_dequantize(q, s, v)
        torch.cuda.synchronize()
        # 6 * 2^127 is past both types: infinite, as the value's conversion is
        w = ref.values4(q, s).to(t)
        assert torch.equal(torch.isnan(v), torch.isnan(w)), t
        assert torch.equal(v[:255], w[:255]), t


@pytest.mark.parametrize("case", [(5, 640, BF, 0, True, False, True), (3, 32832, BF, 0, True, False, True),
                                  (6, 20000, F32, 0, False, False, True), (5, 640, F32, 0, True, False, False),
                                  (64, 8192, BF, 7, True, True, True), (515, 4100, F32, 0, True, True, True)], ids=ident)
def test_a_gate_without_a_norm_behind_and_wide_rows(case):
    test_block_norm(case)
    test_block_norm_backward(case)
