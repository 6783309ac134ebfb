"""The size that kv_cache_move takes at most, for every format and head size
(no GPU): S * heads times a row's pieces, the 16-byte pieces of its codes and
the pieces of its scales (the largest power of two that divides their bytes),
keys and values, is below 2^31."""
import pytest

from test_kv_cpu import L, cache, msg, needs_device  # noqa: F401 (L is a fixture)
from test_kv_tree_cpu import move

MODES = {"nvfp4": (0, 4, 16), "mxfp8": (1, 8, 32), "mxfp4": (2, 4, 32)}


def row_pieces(mode, D):
    _, bits, group = MODES[mode]
    scales = D // group
    return 2 * (D * bits // 128 + scales // (scales & -scales))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("D", range(32, 257, 32))
def test_the_largest_call(L, mode, D):  # noqa: F811
    c, n = cache(mode=MODES[mode][0], heads=1, D=D), row_pieces(mode, D)
    S = (2 ** 31 - 1) // n
    assert needs_device(move(L, c, M=S, S=S))
    assert move(L, c, M=S + 1, S=S + 1) == 2 and f"heads*{n} must" in msg(L)


def test_the_most_pieces():
    assert max((row_pieces(m, D), m, D) for m in MODES for D in range(32, 257, 32)) == (42, "mxfp8", 224)
