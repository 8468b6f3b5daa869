"""The layer classes on 4-bit weights and for a few tokens, without a GPU: which calls
they make, and what they refuse."""
import pytest

torch = pytest.importorskip("torch")
import expert_load_balance_amd as moe  # noqa: E402
from expert_load_balance_amd import layer  # noqa: E402

from test_block_contract import _Elsewhere  # noqa: E402

SHAPE = moe.Shape(4, 128, 8, 2, 128, 4, 2, moe.MOE_BF16)


@pytest.mark.parametrize("bits,gemm", [(8, "moe_grouped_gemm_mx"), (4, "moe_grouped_gemm_mx4")])
def test_weight_bits_choose_the_product(monkeypatch, bits, gemm):
    calls = []
    for name in ("moe_count_plan", "moe_permute_mx", "moe_grouped_gemm_mx", "moe_grouped_gemm_mx4", "moe_combine"):
        monkeypatch.setattr(layer, name, lambda *a, _n=name, **k: calls.append(_n))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    L = layer.MoeLayerMx(SHAPE, "cpu", weight_bits=bits)
    assert L.mx_ws.numel() == (moe.moe_mx_workspace_bytes if bits == 8 else moe.moe_mx4_workspace_bytes)(SHAPE)
    L.err, here = _Elsewhere(0), _Elsewhere(0)
    L.experts(here, here, here, here, *[(here, here)] * 3, stream=0)
    assert calls == ["moe_count_plan", "moe_permute_mx", gemm, "moe_combine"]
    calls.clear()
    with pytest.raises(ValueError, match="current device"):
        L.experts(here, here, _Elsewhere(1), here, *[(here, here)] * 3, stream=0)
    assert calls == []


def test_weight_bits_that_are_none():
    for bits in (0, 2, 16):
        with pytest.raises(ValueError, match="bits"):
            layer.MoeLayerMx(SHAPE, "cpu", weight_bits=bits)


def test_few_refuses_what_it_has_no_layer_for():
    for shape, kw in ((moe.Shape(33, 128, 8, 2, 128, 4, 2, moe.MOE_BF16), {}),
                      (moe.Shape(4, 128, 8, 2, 128, 4, 2, moe.MOE_F32), {}),
                      (moe.Shape(4, 192, 8, 2, 128, 4, 2, moe.MOE_BF16), {}),
                      (moe.Shape(4, 8320, 8, 2, 128, 4, 2, moe.MOE_BF16), {}),
                      (SHAPE, {"shared_F": 64})):
        with pytest.raises(ValueError, match="no layer of this shape"):
            layer.MoeLayerFew(shape, "cpu", **kw)
    with pytest.raises(KeyError):
        layer.MoeLayerFew(SHAPE, "cpu", weights="int8")
    assert layer.MoeLayerFew(moe.Shape(4, 192, 8, 2, 64, 4, 2, moe.MOE_BF16), "cpu", weights="bf16").ws.numel() > 0
