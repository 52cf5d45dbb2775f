"""Which kernel and tile the 16-bit products choose: the sizes that the GPU tests take for a tile reach it,
and every tile that can be chosen is among them."""
import ctypes
import os

import pytest

import routing_permute_mxfp8_amd as rp
from gmm16_cases import FORMS, MANY_ITEMS, cases


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rp.lib_path()):
        from routing_permute_mxfp8_amd import build
        build.build()
    return rp.load()


def plan(lib, form, rows, groups, n, k):
    tile, shared = ctypes.c_int(-1), ctypes.c_int(-1)
    assert lib.moe_grouped_matmul_plan(FORMS.index(form), rows, groups, n, k, ctypes.byref(tile), ctypes.byref(shared)) == 0
    return tile.value, shared.value


@pytest.mark.parametrize("form,tile,shared,rows,groups,n,k", cases())
def test_the_cases_reach_their_tiles(lib, form, tile, shared, rows, groups, n, k):
    assert plan(lib, form, rows, groups, n, k) == (tile, shared)


@pytest.mark.parametrize("form,tile,each,groups,n,k", MANY_ITEMS)
def test_the_cases_of_many_items(lib, form, tile, each, groups, n, k):
    """They reach their tiles, and 256 units of three, two or one blocks at a time have over 64 items for each."""
    assert plan(lib, form, each * groups, groups, n, k)[0] == tile
    up = lambda a, b: -(-a // b)  # noqa: E731
    width, blocks = (256, 1) if tile > 64 else (128, {64: 2, 32: 3}[tile])
    items = groups * (up(n, tile) * up(k, width) if form == "weights" else up(each, tile) * up(n, width))
    assert items > 65 * 256 * blocks


@pytest.mark.parametrize("form", FORMS)
def test_no_tile_without_cases(lib, form):
    """What the planner chooses over a grid of sizes is a tile, shared or not, that has cases."""
    have = {(t, s) for f, t, s, *_ in cases() if f == form}
    sizes = [1, 8, 60, 136, 776, 2056, 7168, 16384]
    for rows in (1, 9, 33, 100, 161, 300, 777, 2100, 8192, 32768):
        for groups in (1, 3, 16, 40, 256):
            for n in sizes:
                for k in sizes:
                    tile, shared = plan(lib, form, rows, groups, n, k)
                    assert tile == 0 and form == "forward" or (tile, shared) in have, (rows, groups, n, k)


def test_refusals(lib):
    a, b = ctypes.c_int(), ctypes.c_int()
    pa, pb = ctypes.byref(a), ctypes.byref(b)
    for args, status in [((3, 4, 1, 8, 8, pa, pb), 1), ((-1, 4, 1, 8, 8, pa, pb), 1), ((0, 4, 1, 8, 8, None, pb), 1),
                         ((0, 4, 1, 8, 8, pa, None), 1), ((0, -1, 1, 8, 8, pa, pb), 2), ((1, 4, 0, 8, 8, pa, pb), 2),
                         ((2, 4, 1, 0, 8, pa, pb), 2), ((2, 4, 1, 8, (1 << 20) + 1, pa, pb), 2)]:
        assert lib.moe_grouped_matmul_plan(*args) == status and lib.moe_last_error().decode()
