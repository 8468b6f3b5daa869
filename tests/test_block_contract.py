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
