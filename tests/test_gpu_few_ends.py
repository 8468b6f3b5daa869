"""moe_few_layer at the ends of its ranges: the widest shared expert, values of h next to
and past the largest bf16."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd.layer import MoeLayerFew  # noqa: E402

import step_ref as ref  # noqa: E402
from test_gpu_few import BF, DEV, blocks, check, gen, randn  # noqa: E402

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


@pytest.mark.parametrize("form", ["bf16", "mx8", "mx4"])
@pytest.mark.parametrize("column", [5, 66])
def test_h_next_to_and_past_the_largest_value(form, column):
    """One column of h is 1.996 * 2^127, which float32 holds and bf16's rounding makes
    infinite, or twice that, which is infinite in float32; the others are 0. Every product
    and sum is exact but for silu's quotient (2^-22 of it at most) and out's rounding."""
    T, H, F = 5, 128, 128
    x = torch.zeros(T, H)
    x[:, 0] = torch.tensor([1.0, 1.0, -1.0, 1.0, -1.0])
    x[:, 1] = torch.tensor([1.328125, 1.328125, -1.328125, -1.328125, -1.328125])   # u 2^121 times 1.996 or 2^-8
    x[:, 32] = torch.tensor([1.0, 2.0, 1.0, 1.0, 2.0])                               # g 64 or 128
    gate, up, down = torch.zeros(1, F, H), torch.zeros(1, F, H), torch.zeros(1, H, F)
    gate[0, column, 32] = 64.0
    up[0, column, 0], up[0, column, 1] = 2.0 ** 121, 0.75 * 2.0 ** 121
    down[0, :, column] = 2.0 ** -100
    down[0, ::3, column] = -2.0 ** -101
    w = [blocks(form, v.to(DEV)) for v in (gate, up, down)]
    L = MoeLayerFew(moe.Shape(T, H, 1, 1, F, 1, 0, moe.MOE_BF16), DEV, weights=form)
    L.forward(x.to(DEV).to(BF), torch.zeros(1, H, dtype=BF, device=DEV), None, *w)
    torch.cuda.synchronize()
    h = x[:, 32].double() * 64 * (x[:, 0].double() + 0.75 * x[:, 1].double()) * 2.0 ** 121
    want = (h[:, None] * down[0, :, column].double()).to(DEV)
    fits = torch.tensor([0, 2, 3], device=DEV)
    assert h[0] == 1.99609375 * 2.0 ** 127 and float(h[:1].to(BF)) == float("inf")
    ref.check(L.out[fits], (want[fits], want[fits].abs() * 2.0 ** -22), "out", BF)
    for t in (1, 4):
        assert torch.equal(L.out[t].float(), torch.sign(want[t]).float() * float("inf")), t


@pytest.mark.parametrize("form,lowest,highest", [("mx8", 3, 246), ("mx4", 0, 252)])
def test_scales_at_the_ends_of_their_range(form, lowest, highest):
    """W_down with a scale byte of its own in every row (2^-124 to 2^119 for 8-bit codes, 2^-127
    to 2^125 for 4-bit ones widen to bf16 exactly), times an h of about 2^108, 2^8 and 2^-92: the
    products that float32 holds come out as the layer's do in general (bounds as in step_ref's
    swiglu, h exact)."""
    T, H, F = 3, 256, 256
    g = gen(1)
    x = torch.zeros(T, H)
    x[:, 0], x[:, 32] = 1, torch.tensor([2.0 ** 100, 1.0, 2.0 ** -100])
    gate, up = (torch.zeros(1, F, H, device=DEV) for _ in range(2))
    gate[0, :, 0] = 64
    up[0, :, 32] = torch.randint(1, 7, (F,), generator=g, device=DEV) * torch.sign(randn(g, F))
    q = torch.randint(0, 256, (1, H, F if form == "mx8" else F // 2), generator=g, device=DEV)
    if form == "mx8":
        q = torch.where(q % 128 == 127, q - 1, q)          # (the codes that are NaN)
    s = torch.arange(H, device=DEV).clamp(max=254).to(torch.uint8)[None, :, None].expand(1, H, F // 32).contiguous()
    w = [blocks(form, gate), blocks(form, up), (q.to(torch.uint8), s)]
    L = MoeLayerFew(moe.Shape(T, H, 1, 1, F, 1, 0, moe.MOE_BF16), DEV, weights=form)
    x = x.to(DEV).to(BF)
    L.forward(x, torch.zeros(1, H, dtype=BF, device=DEV), None, *w)
    torch.cuda.synchronize()
    G, U, D = (ref.whole(m, 0) for m in w)
    h = (x.double() @ G.t()) * (x.double() @ U.t())         # silu(64) is 64 but for 2^-90 of it
    want, size = h @ D.t(), h.abs() @ D.abs().t()
    byte = torch.arange(H, device=DEV)
    inside = (byte >= lowest) & (byte <= highest) & (size < 2.0 ** 126) & (size > 2.0 ** -100)
    assert bool(inside.any(0)[lowest:highest + 1].all())
    tol = (F / 128 + 24) * 2.0 ** -22 * size
    ref.check(L.out[inside], (want[inside], tol[inside]), form, BF)
