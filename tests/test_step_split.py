"""The split of the down projection's K in moe_few_layer (csrc/split.h) at every size that
the host checks let through, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

import expert_load_balance_amd as moe

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_load_balance_amd", "csrc")
UNIT = {moe.MOE_W_BF16: 64, moe.MOE_W_MX8: 128, moe.MOE_W_MX4: 256}
PART = 4096   # values of K of a part; half of it where entries have two tiles of rows


@pytest.fixture(scope="module")
def part_begin(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    src, lib = str(d / "split.cpp"), str(d / "split.so")
    with open(src, "w") as f:
        f.write('#include "split.h"\nextern "C" int part_begin(int p, int u, int n) { return moe::part_begin(p, u, n); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib])
    return ctypes.CDLL(lib).part_begin


def widest(form, H):
    """The widest shared expert of a layer of width H that has a workspace."""
    shape, step = moe.Shape(1, H, 1, 1, 128, 1, 0, moe.MOE_BF16), 64 if form == moe.MOE_W_BF16 else 128
    lo, hi = 1, (1 << 31) // step // H + 1   # of the step: taken, refused
    assert moe.moe_few_workspace_bytes(shape, form, hi * step) == 0
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if moe.moe_few_workspace_bytes(shape, form, mid * step) else (lo, mid)
    return lo * step


@pytest.mark.parametrize("form", sorted(UNIT))
@pytest.mark.parametrize("tiles", [1, 2])
def test_the_parts_cover_k(part_begin, form, tiles):
    top = widest(form, 64 if form == moe.MOE_W_BF16 else 128)
    assert top >= (1 << 24) - 128
    for K in (128, 4096, 4224, 147456, 1 << 23, top // 3 // 128 * 128, top - 128, top):
        units, parts = -(-K // UNIT[form]), -(-K * tiles // PART)
        at = [part_begin(p, units, parts) for p in range(parts + 1)]
        assert at == [p * units // parts for p in range(parts + 1)], K
        # a wave has registers for an eighth of the longest part
        assert at[0] == 0 and at[-1] == units
        assert max(b - a for a, b in zip(at, at[1:])) <= -(-PART // tiles // UNIT[form]), K
