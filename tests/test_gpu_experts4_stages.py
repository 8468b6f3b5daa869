"""The experts on 4-bit weights where small tiles cut K or turn its order, and K is an odd
multiple of 128: the last stage of 256 values is half a one, in a part that does not begin
at 0, or among the others. (Eight stages and more, 1920 values, may be cut; a number of
stages that is a multiple of four, as of 1920 and 2944 values, is turned.)"""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerMx  # noqa: E402

from test_gpu_block import DEV, gen, quantized, randn, say  # noqa: E402
from test_gpu_experts4 import check, run, weights4  # noqa: E402

pytestmark = pytest.mark.gpu


# experts and rows of each: few tiles, cut along K, of 32, 64 and 128 rows and with whole
# ones of 256; more tiles than workgroups, of every size, most of them whole
@pytest.mark.parametrize("E,rows", [(2, 3), (2, 50), (2, 100), (3, 300), (40, 12), (40, 45), (40, 100)])
@pytest.mark.parametrize("H,F", [(1920, 2176), (2176, 2944), (2944, 1920), (896, 1920)])
def test_half_a_stage(H, F, E, rows):
    T = E * rows
    say("experts_mx4 stages", H, F, E, rows)
    g = gen(H + F + T)
    L = MoeLayerMx(moe.Shape(T, H, E, 1, F, 1, 0, moe.MOE_BF16), DEV, weight_bits=4)
    xq, xs = quantized(randn(g, T, H) * torch.exp(randn(g, H)))
    ids = torch.randperm(T, generator=g, device=DEV).remainder(E).to(torch.int32)[:, None]
    w = torch.ones(T, 1, device=DEV)
    wts = weights4(g, E, F, H)
    run(L, xq, xs, ids, w, wts)
    check(L, xq, xs, ids, wts)
    want, on, last = L.out.clone(), ids[:, 0] == 0, ids[:, 0] == E - 1
    # NaN scales where a row's last ones are read together with the next row's first: rows of
    # W_down of the first expert, the rows of W_gate and W_up behind the last but one, tokens
    wts[2][1][0, 70:73] = 255
    wts[0][1][E - 1, 0], wts[1][1][E - 1, 0] = 255, 255
    xs[::7] = 255
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[::7] = True
    bad |= last
    run(L, xq, xs, ids, w, wts)
    assert bool(torch.isnan(L.out[bad]).all())
    fine, cols = ~bad & ~on, [c for c in range(H) if not 70 <= c < 73]
    assert torch.equal(L.out[fine], want[fine])
    fine = ~bad & on
    assert bool(torch.isnan(L.out[fine][:, 70:73]).all()) and torch.equal(L.out[fine][:, cols], want[fine][:, cols])
