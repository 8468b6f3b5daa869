"""The experts on 4-bit weights where the scales of h pass 2^32 bytes."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402

import block_ref  # noqa: E402
from test_gpu_block import BF, DEV, gen, quantized, randn, say  # noqa: E402
from test_gpu_experts4 import as_eights, weights4  # noqa: E402

pytestmark = pytest.mark.gpu


def test_scales_of_h_of_2_32_bytes():
    """8 experts of 2^20 rows each, 16384 columns of h: 2^32 scales and 137 GB of codes, in
    tiles of 128 rows. The workspace of the bf16 GEMM would be twice that, so the calls are
    the ones that need none of it."""
    T, H, E, k, F = 1 << 20, 128, 8, 8, 16384
    shape = moe.Shape(T, H, E, k, F, 1, 0, moe.MOE_BF16)
    N = shape.N
    need = moe.moe_mx4_workspace_bytes(shape)
    if torch.cuda.mem_get_info()[0] < need + (12 << 30):
        pytest.skip("not enough memory free")
    say("experts_mx4", T, H, E, k, F, "workspace", need)
    g = gen(1)
    xq, xs = quantized(randn(g, T, H))
    ids = torch.arange(k, dtype=torch.int32, device=DEV).expand(T, k).contiguous()
    wts = weights4(g, E, F, H)

    def ints(n):
        return torch.zeros(n, dtype=torch.int32, device=DEV)

    counts, offsets, eidx, load, err, plan = ints(E), ints(E + 1), ints(N), ints(1), ints(1), ints(moe.plan_layout_total(shape))
    dest, src = ints(N), ints(N)
    a, a_s = torch.empty((N, H), dtype=torch.uint8, device=DEV), torch.empty((N, H // 32), dtype=torch.uint8, device=DEV)
    y = torch.full((N, H), float("nan"), dtype=BF, device=DEV)
    moe.moe_count_noalloc(shape, ids, counts, offsets, eidx, load, err)
    moe.moe_plan(shape, counts, plan)
    moe.moe_permute_mx(shape, xq, xs, ids, eidx, plan, a, a_s, dest, src)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    try:
        moe.moe_grouped_gemm_mx4(shape, a, a_s, plan, *wts, y, ws)
        torch.cuda.synchronize()
    finally:
        del ws
        torch.cuda.empty_cache()
    assert int(err.item()) == 0 and counts.tolist() == [T] * E
    wide = tuple(as_eights(w) for w in wts)
    for lo, hi in ((0, 300), (511, 513), (N // 2 - 150, N // 2 + 150), (N - 300, N)):
        rows = torch.arange(lo, hi, device=DEV)
        want, tol = block_ref.experts(block_ref.values(a[rows], a_s[rows]), a_s[rows], rows // T, *wide)
        got = y[rows].double()
        bad = ~((got - want).abs() <= (want.abs() + tol) * block_ref.HALF[BF] + tol + 1e-30)
        assert not bool(bad.any()), (lo, int(bad.sum()))
        # (a value's own rounding, and codes of h that are the neighbour's: see test_gpu_experts4)
        assert float((got - want).norm() / want.norm()) <= 0.0035, lo
