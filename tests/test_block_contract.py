"""include/moe_block.h without a GPU: calls that its text allows, and what the
binding refuses before anything is launched."""
import ctypes
import os

import pytest

import expert_load_balance_amd as moe
from expert_load_balance_amd.block import GradT

EINVAL = 1
P = ctypes.c_void_p(4096)   # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        pytest.fail("libmoe.so is not built: run `python -m expert_load_balance_amd.build`")
    return moe.load()


def test_grad_workspace_bytes_reads_the_counts_only(lib):
    """A list that holds the counts and whatever the memory held before."""
    counts = (0, 1, 16384, 16385, (1 << 40) - 1)
    plain, stale = (GradT * len(counts))(), (GradT * len(counts))()
    ctypes.memset(stale, 0xA5, ctypes.sizeof(stale))
    for i, n in enumerate(counts):
        plain[i].count = stale[i].count = n
    need = lib.moe_grad_workspace_bytes(len(counts), plain)
    assert need > 0 and lib.moe_grad_workspace_bytes(len(counts), stale) == need
    stale[2].count = 1 << 40
    assert lib.moe_grad_workspace_bytes(len(counts), stale) == 0
    stale[2].count = -1
    assert lib.moe_grad_workspace_bytes(len(counts), stale) == 0
    # the calls themselves still refuse a type that is none
    stale[2].count = 16384
    assert lib.moe_grad_norm(len(counts), stale, P, P, P, need, None) == EINVAL
    assert lib.moe_grad_clip(len(counts), stale, 1.0, P, None) == EINVAL


class _Elsewhere:
    """Stands for a tensor of device `index`."""

    def __init__(self, index):
        self.index, self.device = index, f"cuda:{index}"

    def get_device(self):
        return self.index

    def zero_(self):
        return self


@pytest.mark.parametrize("which", ["ids", "w", "shared_y", "err", "w_router", "bias"])
def test_layer_refuses_another_device_before_any_launch(monkeypatch, which):
    """The first kernels of the 8-bit layer read ids and write the layer's own
    buffers: what lies on another device than the current one is refused
    before them, not by a later call of the sequence."""
    torch = pytest.importorskip("torch")
    from expert_load_balance_amd import layer

    calls = []
    for name in ("moe_rmsnorm", "moe_router", "moe_count_plan", "moe_permute_mx", "moe_grouped_gemm_mx", "moe_combine"):
        monkeypatch.setattr(layer, name, lambda *a, _n=name, **k: calls.append(_n))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: __import__("contextlib").nullcontext())
    L = layer.MoeLayerMx(moe.Shape(4, 128, 8, 2, 128, 4, 2, moe.MOE_BF16), "cpu")
    L.err = _Elsewhere(1 if which == "err" else 0)
    at = {n: _Elsewhere(1 if n == which else 0) for n in ("ids", "w", "shared_y", "w_router", "bias")}
    here, wts = _Elsewhere(0), [(_Elsewhere(0), _Elsewhere(0))] * 3
    if which in ("ids", "w", "shared_y", "err"):
        with pytest.raises(ValueError, match="current device"):
            L.experts(here, here, at["ids"], at["w"], *wts, shared_y=at["shared_y"], stream=0)
        assert calls == []
    if which in ("w_router", "bias", "err"):
        with pytest.raises(ValueError, match="current device"):
            L.forward(here, None, here, 1e-6, at["w_router"], at["bias"], *wts, stream=0)
        assert calls == []
    # all in place: the sequence runs, with and without a shared expert's rows
    L.err = L.ids = L.w = _Elsewhere(0)
    for shared in (None, _Elsewhere(0)):
        calls.clear()
        L.experts(here, here, here, here, *wts, shared_y=shared, stream=0)
        assert calls == ["moe_count_plan", "moe_permute_mx", "moe_grouped_gemm_mx", "moe_combine"]
    calls.clear()
    L.forward(here, None, here, 1e-6, here, None, *wts, stream=0)
    assert calls[:3] == ["moe_rmsnorm", "moe_router", "moe_count_plan"] and len(calls) == 6
