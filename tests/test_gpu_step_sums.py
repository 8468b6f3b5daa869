"""The sums over rows of moe_block_norm_backward where a workgroup takes several rows, on
every kernel: all terms are positive, so that the bound is a share of the sum and smaller
than what any one workgroup adds to it."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402

import step_ref as ref  # noqa: E402
from test_gpu_step import ALPHA, BF, DEV, EPS, F32, gen, guarded, say, shape_of  # noqa: E402

pytestmark = pytest.mark.gpu


def chains(T, H, t, rows):
    """Adds in turn of a weight's gradient and of a row of gates', and the workgroups that
    share a weight's: a workgroup takes whole parts, a part every n-th row of a group, and
    sixteen threads add the workgroups' (or a group's parts') sums, every sixteenth each."""
    waves = -(-H // (8 if t == BF else 4) // 64)
    G = 256 * (1 if waves > 8 else 2 if waves > 4 else 4)
    group = rows if 0 < rows < T else T
    groups = -(-T // group)
    per = min(-(-G // groups), group)
    parts = groups * per
    grid = min(parts, G)
    part_rows = -(-group // per)
    mine = -(-parts // grid)
    return mine * (part_rows + 1) + -(-grid // 16) + 16, part_rows + -(-per // 16) + 16, grid


# T, H, type, rows of the gate (0: a value a token)
CASES = [
    (600, 20000, F32, 0), (600, 20000, F32, 1), (600, 20000, F32, 40), (600, 20000, F32, 600),       # three passes
    (600, 32832, BF, 0), (600, 32832, BF, 1), (600, 32832, BF, 40), (600, 32832, BF, 600),
    (700, 12288, BF, 0), (700, 12288, BF, 1), (700, 12288, BF, 37), (700, 7168, F32, 700),           # two vectors a thread
    (700, 4160, BF, 1), (700, 4160, BF, 37), (700, 4160, BF, 700), (2100, 4160, BF, 5),              # one, nine to sixteen waves
    (700, 7168, BF, 0), (700, 7168, BF, 1), (700, 7168, BF, 37), (700, 7168, BF, 700), (1400, 4096, F32, 3),
    (2100, 2304, BF, 1), (2100, 2304, BF, 64), (777, 1540, F32, 37),                                 # five to eight
    (5000, 512, BF, 1), (5000, 512, BF, 3), (5000, 520, F32, 2500),                                  # one to three
    ((1 << 21) + 5, 64, BF, 3), ((1 << 21) + 5, 64, BF, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c[0]}H{c[1]}{'bf16' if c[2] == BF else 'f32'}g{c[3]}")
def test_sums_over_rows(case):
    T, H, t, rows = case
    say("block_norm_backward sums", case)
    g, shape = gen(T + H + rows), shape_of(T, H, t)

    def positive(low, *size):
        return (low + torch.rand(size, generator=g, device=DEV)).to(t)

    # d >= 8 - rstd_pre * shat * mean: s is 0.4 and more, so rstd_pre <= 2.5, shat <= 1.5 times
    # that and the mean below 2.5 at the very most
    x, r, dy, ds = positive(0.5, T, H), positive(0.5, T, H), positive(0.5, T, H), positive(12, T, H)
    w1, w2 = positive(0.5, H), positive(0.5, H)
    gate = positive(0.5, T) if rows == 0 else positive(0.5, -(-T // rows), H)
    s, r1, r2 = torch.empty_like(x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    kw = dict(alpha=ALPHA, w_post=w1, gate=gate, gate_rows=rows, w_pre=w2)
    moe.moe_block_norm(shape, x, EPS, residual=r, s=s, rstd_post=r1, rstd_pre=r2, **kw)
    (dx, a_ok), (dr, b_ok), (dw1, c_ok), (dw2, d_ok) = guarded(T * H, t), guarded(T * H, t), guarded(H, F32), guarded(H, F32)
    dg, e_ok = guarded(gate.numel(), F32)
    ws, f_ok = guarded(moe.moe_block_norm_backward_workspace_bytes(shape, rows), torch.uint8)
    ws.fill_(0xFF)
    moe.moe_block_norm_backward(shape, x, r1, dy, ds, dx, ws, s=s, rstd_pre=r2, dresidual=dr, dw_post=dw1, dw_pre=dw2,
                                dgate=dg, **kw)
    torch.cuda.synchronize()
    assert a_ok() and b_ok() and c_ok() and d_ok() and e_ok() and f_ok()
    want = ref.block_norm_bwd(x, r1, s, r2, ALPHA, w1, gate, rows, w2, dy, ds)
    of_weights, of_gate, grid = chains(T, H, t, rows)
    for name, got, n, length in (("dw_post", dw1, T, of_weights), ("dw_pre", dw2, T, of_weights),
                                 ("dgate", dg.view(gate.shape), min(rows, T), of_gate)):
        v, tol = want[name]
        assert bool((v > 0).all())
        if name != "dgate" or rows:                # the chain that the sum has, in the place of all rows in turn
            tol = tol + (length - n) * ref.U * v
            # and finer than a workgroup's share of a weight's sum
            assert name == "dgate" or bool((tol <= v / grid / 2).all())
        ref.check(got, (v, tol), name)
    ref.check(dx.view(T, H), want["dx"], "dx", t)
    ref.check(dr.view(T, H), want["dresidual"], "dresidual", t)
