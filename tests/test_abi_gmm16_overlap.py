"""16-bit products whose output lies over the group offsets, or whose workspace lies over another tensor, are
refused on the host, before any launch."""
import ctypes

import pytest

from test_abi_dense import lib, product, wgrad  # noqa: F401  (lib: the fixture)

GB = 1 << 30
ROWS, GROUPS, N, K = 640, 4, 61, 259   # odd rows: copies of both operands in the workspace
APART = {"x": GB, "w": 2 * GB, "off": 3 * GB, "out": 4 * GB, "work": 5 * GB}
OFF_BYTES = 4 * (GROUPS + 1)


def need(lib, form):  # noqa: F811
    b = ctypes.c_size_t()
    if form is wgrad:
        assert lib.moe_grouped_matmul_wgrad_workspace_size(ROWS, GROUPS, N, K, ctypes.byref(b)) == 0
    else:
        assert lib.moe_grouped_matmul_workspace_size(ROWS, GROUPS, N, K, 0, ctypes.byref(b)) == 0
    assert b.value > 4096
    return b.value


def refused(lib, form, kw):  # noqa: F811
    assert form(lib, rows=ROWS, groups=GROUPS, n=N, k=K, **{**APART, **kw}) == 1
    return "overlaps" in lib.moe_last_error().decode()


@pytest.mark.parametrize("form", [product, wgrad])
def test_the_offsets(lib, form):  # noqa: F811
    for at in (APART["off"], APART["off"] + OFF_BYTES - 2, APART["off"] - 2):
        assert refused(lib, form, dict(out=at))


@pytest.mark.parametrize("form", [product, wgrad])
@pytest.mark.parametrize("name", ["x", "w", "off", "out"])
def test_the_workspace(lib, form, name):  # noqa: F811
    last = need(lib, form) // 4 * 4 - 4   # a tensor that begins in the workspace's last bytes
    for kw in ({"work": APART[name]}, {name: APART["work"] + last}):
        assert refused(lib, form, kw), kw
