"""The operators of include/moe_step.h at sizes whose offsets pass 31 and 32 bits, more
rows than a launch takes, and the most assignments of the layer for a few tokens."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402

import step_ref as ref  # noqa: E402
from test_gpu_few import check as check_few, layer  # noqa: E402
from test_gpu_step import ALPHA, BF, DEV, EPS, F32, gen, randn, shape_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [(32, 128, 256, 64, 128, 128, "mx4"), (32, 64, 256, 64, 64, 0, "bf16"),
                                  (17, 128, 64, 64, 256, 0, "mx8")], ids=str)
def test_few_most_assignments(case):
    L, *inputs = layer(case)
    L.ws.fill_(0xFF)
    L.forward(*inputs[:3], *inputs[3], inputs[4])
    torch.cuda.synchronize()
    check_few(L, *inputs, str(case))


def test_few_projection_above_2_31_bytes():
    """One expert of 8192 x 147456 in bf16: 2.4 GB a projection, 36 parts of the down
    projection's K."""
    case = (2, 8192, 1, 1, 147456, 0, "bf16")
    print("[case]", case, flush=True)
    L, *inputs = layer(case)
    L.forward(*inputs[:3], *inputs[3], inputs[4])
    torch.cuda.synchronize()
    check_few(L, *inputs, str(case))


def test_mx4_more_than_2_32_values():
    rows, cols = (1 << 20) + 3, 4128
    print("[case]", rows, cols, flush=True)
    x = torch.empty((rows, cols), dtype=BF, device=DEV).normal_(generator=gen(1))
    q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
    s = torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV)
    moe.moe_mx4_quantize(x, q, s)
    back = torch.empty_like(x)
    moe.moe_mx4_dequantize(q, s, back)
    torch.cuda.synchronize()
    for a in (0, rows // 2, (1 << 32) // cols - 32, rows - 64):
        part = slice(a, a + 64)
        codes, scales = ref.codes4(x[part].double())
        assert torch.equal(s[part], scales) and torch.equal(ref.unpack4(q[part]), codes), a
        assert torch.equal(back[part].double(), ref.values4(q[part], s[part])), a


def test_block_norm_more_rows_than_a_launch():
    T, H = (1 << 21) + 5, 64
    print("[case]", T, H, flush=True)
    g, shape = gen(2), shape_of(T, H, BF)
    x, r, dy = (randn(g, T, H).to(BF) for _ in range(3))
    w1, w2, gate = (1 + 0.2 * randn(g, H)).to(BF), (1 + 0.2 * randn(g, H)).to(BF), randn(g, -(-T // 3), H).to(BF)
    s, y, dx, dr = (torch.full_like(x, float("nan")) for _ in range(4))
    r1, r2, dw1, dw2 = (torch.full((n,), float("nan"), device=DEV) for n in (T, T, H, H))
    dg = torch.full(gate.shape, float("nan"), device=DEV)
    kw = dict(alpha=ALPHA, w_post=w1, gate=gate, gate_rows=3, w_pre=w2)
    moe.moe_block_norm(shape, x, EPS, residual=r, s=s, y=y, rstd_post=r1, rstd_pre=r2, **kw)
    ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(shape, 3), dtype=torch.uint8, device=DEV)
    moe.moe_block_norm_backward(shape, x, r1, dy, None, dx, ws, s=s, rstd_pre=r2, dresidual=dr, dw_post=dw1, dw_pre=dw2,
                                dgate=dg, **kw)
    torch.cuda.synchronize()
    want, tol, _ = ref.block_norm(x, r, ALPHA, w1, gate, 3, w2, EPS)
    ref.check(s, (want, tol), "s", BF)
    ref.check(y, ref.pre_norm(s, w2, EPS)[:2], "y", BF)
    got = dict(dx=dx, dresidual=dr, dw_post=dw1, dw_pre=dw2, dgate=dg)
    for name, bound in ref.block_norm_bwd(x, r1, s, r2, ALPHA, w1, gate, 3, w2, dy, None).items():
        ref.check(got[name], bound, name, BF if name in ("dx", "dresidual") else None)


def test_block_norm_more_than_2_31_values():
    """Rows behind element 2^31, forward and backward, with one array as dy and ds."""
    T, H = 131080, 16416
    print("[case]", T, H, flush=True)
    g, shape = gen(3), shape_of(T, H, F32)
    x = torch.empty((T, H), device=DEV).normal_(generator=g)
    dy = torch.empty((T, H), device=DEV).normal_(generator=g)
    w1, w2, gate = 1 + 0.2 * randn(g, H), 1 + 0.2 * randn(g, H), randn(g, T)
    s, dx = torch.empty_like(x), torch.empty_like(x)
    r1, r2, dg = (torch.empty(T, device=DEV) for _ in range(3))
    kw = dict(alpha=ALPHA, w_post=w1, gate=gate, gate_rows=0, w_pre=w2)
    moe.moe_block_norm(shape, x, EPS, residual=x, s=s, rstd_post=r1, rstd_pre=r2, **kw)
    ws = torch.empty(moe.moe_block_norm_backward_workspace_bytes(shape, 0), dtype=torch.uint8, device=DEV)
    moe.moe_block_norm_backward(shape, x, r1, dy, dy, dx, ws, s=s, rstd_pre=r2, dgate=dg, **kw)
    torch.cuda.synchronize()
    for a in (0, 65536, (1 << 31) // H - 8, T - 16):
        p = slice(a, a + 16)
        want, tol, _ = ref.block_norm(x[p], x[p], ALPHA, w1, gate[p], 0, w2, EPS)
        ref.check(s[p], (want, tol), "s", F32)
        out = ref.block_norm_bwd(x[p], r1[p], s[p], r2[p], ALPHA, w1, gate[p], 0, w2, dy[p], dy[p])
        ref.check(dx[p], out["dx"], "dx", F32)
        ref.check(dg[p], out["dgate"], "dgate")
