"""The sizes that the GPU tests of the 4-bit products name still take every way
of cutting one (no GPU): few rows in each of its forms, each tile, for each
kind of x, plain and gated."""
import ctypes
import os

import pytest

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_tile_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

FEW = [(0, 1, 2, 2), (0, 1, 2, 4), (0, 1, 4, 4), (0, 2, 4, 4)]
TILES = {0: [1, 2, 4, 5], 3: [1, 2, 3, 5]}


def _choice(M, N, K, E, dtype, gated):
    import moe_expert_tile_amd as m
    out = (ctypes.c_int32 * 4)()
    d = m.moe_mx_linear_desc(M, E, N, K, dtype, 0, m.ACT_SWIGLU if gated else m.ACT_NONE)
    # moe::mx_choice, an internal symbol of the library
    m._lib._ZN3moe9mx_choiceERK18moe_mx_linear_descPi(ctypes.byref(d), out)
    return tuple(out)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [0, 3])
def test_every_cut_is_named(dtype, gated):
    from test_gpu_mx import CUTS, SIZES
    seen = {_choice(*s, dtype, gated) for s in SIZES + CUTS}
    for c in FEW + [(t, 0, 0, 0) for t in TILES[dtype]]:
        assert c in seen, (c, sorted(seen))


def test_every_size_has_a_cut():
    for M in (0, 1, 1 << 26):
        for E in (1, 1024):
            for N, K in ((1, 32), (1 << 20, 1 << 20)):
                assert _choice(M, N, K, E, 0, False)[0] in (0, 1, 2, 4, 5)
                assert _choice(M, N, K, E, 3, True)[0] in (0, 1, 2, 3, 5)
