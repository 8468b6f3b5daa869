"""moe_few_layer at the ends of its ranges: the widest shared expert."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerFew  # noqa: E402

from test_gpu_few import BF, DEV, check, gen, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2, 17])
def test_the_widest_shared_expert(T):
    """A shared expert of 2^25 - 64 on 64 channels, its down projection's K in 8192 parts
    or, with two tiles of rows to an entry, 16384. Each output takes eight columns of h,
    spread over all of them; the other weights are zeros, which add nothing and round
    nothing, so that the float64 form of those columns alone is the layer's."""
    H, F, SF = 64, 64, (1 << 25) - 64
    print("[case]", T, SF, flush=True)
    g = gen(T)
    x = randn(g, T, H).to(BF)
    wr, bias = randn(g, 1, H).to(BF), torch.zeros(1, device=DEV)
    w = [((randn(g, 1, *s) * 0.125).to(BF), None) for s in ((F, H), (F, H), (H, F))]
    gate, up = (torch.empty((1, SF, H), dtype=BF, device=DEV).normal_(0, 0.125, generator=g) for _ in range(2))
    down = torch.zeros((1, H, SF), dtype=BF, device=DEV)
    at = torch.linspace(0, SF - 1, 8 * H, dtype=torch.float64, device=DEV).round().long()
    few_down = torch.zeros((1, H, 8 * H), dtype=BF, device=DEV)
    few_down[0, torch.arange(8 * H, device=DEV) % H, torch.arange(8 * H, device=DEV)] = randn(g, 8 * H).to(BF)
    down[:, :, at] = few_down
    L = MoeLayerFew(moe.Shape(T, H, 1, 1, F, 1, 0, moe.MOE_BF16), DEV, weights="bf16", shared_F=SF)
    L.ws.fill_(0xFF)
    L.forward(x, wr, bias, *w, [(gate, None), (up, None), (down, None)])
    torch.cuda.synchronize()
    check(L, x, wr, bias, w, [(gate[:, at], None), (up[:, at], None), (few_down, None)], f"T {T}")
