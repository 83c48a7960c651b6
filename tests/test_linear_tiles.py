"""The sizes that the GPU tests of the dense product name for its tiles still
choose them (no GPU): each tile, whole and split along K, in each direction."""
import ctypes
import os

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_tile_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

FEW, T64, T128, T256, WIDE = range(5)


def _cut(what, M, N, K, act="none"):
    """(tile, split) of a product, from the library's own choice."""
    import moe_expert_tile_amd as m
    cuts = (ctypes.c_int32 * 6)()
    d = m.moe_linear_desc(M, N, K, 0, 0, m.ACT_SWIGLU if what == "gated" else m.ACT_NONE, 0)
    # moe::linear_cuts, an internal symbol of the library
    m._lib._ZN3moe11linear_cutsERK15moe_linear_descPi(ctypes.byref(d), cuts)
    i = {"fwd": 0, "gated": 0, "dx": 1, "dw": 2}[what]
    return cuts[2 * i], cuts[2 * i + 1] > 1


def test_every_tile_whole_and_split_is_named():
    from test_gpu_linear import EACH_TILE, SIZES
    seen = {(what,) + _cut(what, M, N, K) for what, M, N, K in EACH_TILE}
    for what in ("fwd", "gated", "dx", "dw"):
        for tile in (T64, T128, T256, WIDE):
            for split in (False, True):
                assert (what, tile, split) in seen, (what, tile, split)
    few = {(what,) + _cut(what, M, N, K) for M, N, K in SIZES for what in ("fwd", "gated")}
    for what in ("fwd", "gated"):
        for split in (False, True):
            assert (what, FEW, split) in few, (what, split)


def test_the_epilogue_sizes_take_every_tile():
    from test_gpu_linear_epilogue import GATED, SIZES
    for whole8 in (False, True):
        seen = {_cut("fwd", M, N, K) for M, N, K in SIZES if (N % 8 == 0) == whole8}
        assert seen == {(t, s) for t in (T64, T128, T256, WIDE) for s in (False, True)}, whole8
    seen = {_cut("gated", M, N, K) for M, N, K in GATED}
    assert seen == {(t, s) for t in (T64, T128, T256, WIDE) for s in (False, True)}
