"""Calls of the norm and its gradient whose outputs would overwrite each other, or an input before it is read,
are refused on the host, before any launch."""
import pytest

from test_abi_dense import lib, norm, norm_back  # noqa: F401  (lib: the fixture)

ROWS, COLS = 40, 64
MB = 1 << 20
ALL = 2 * ROWS * COLS   # bytes of the bf16 rows
NAMES = ("x", "res", "w", "y", "h", "rstd", "codes", "scales")
APART = {name: (i + 1) * MB for i, name in enumerate(NAMES)}
BACK_NAMES = ("g", "h", "gh", "w", "rstd", "gx", "gw", "work")
BACK_APART = {name: (i + 1) * MB for i, name in enumerate(BACK_NAMES)}


@pytest.mark.parametrize("name,at", [
    ("y", APART["h"]), ("y", APART["h"] + ALL - 2), ("y", APART["h"] - ALL + 2), ("h", APART["codes"]), ("h", APART["scales"]),
    ("rstd", APART["y"]), ("rstd", APART["h"] + ALL - 4), ("rstd", APART["codes"] + ROWS * COLS - 4), ("codes", APART["scales"]),
    ("y", APART["x"] + 2), ("y", APART["x"] - 2), ("h", APART["res"] + 2 * COLS), ("y", APART["w"]), ("y", APART["w"] + 2 * COLS - 2),
    ("codes", APART["x"]), ("codes", APART["res"] + 8), ("scales", APART["x"] + ALL - 1), ("rstd", APART["x"]), ("rstd", APART["w"]),
    ("scales", APART["rstd"] + 4 * ROWS - 1),
])
def test_norm(lib, name, at):  # noqa: F811
    assert norm(lib, rows=ROWS, cols=COLS, **{**APART, name: at}) == 1
    assert "overlaps" in lib.moe_last_error().decode()


def test_both_in_one_input(lib):  # noqa: F811
    """y and h may each take an input's place, but not the same one."""
    both = {**APART, "y": APART["x"], "h": APART["x"]}
    assert norm(lib, rows=ROWS, cols=COLS, **both) == 1 and "overlaps" in lib.moe_last_error().decode()


@pytest.mark.parametrize("name,at", [
    ("gx", BACK_APART["g"] + 2), ("gx", BACK_APART["h"] - 2), ("gx", BACK_APART["gh"] + 2 * COLS), ("gx", BACK_APART["w"]),
    ("gx", BACK_APART["rstd"]), ("gx", BACK_APART["gw"]), ("gx", BACK_APART["work"]), ("gw", BACK_APART["g"]),
    ("gw", BACK_APART["w"]), ("gw", BACK_APART["rstd"] + 4 * ROWS - 4), ("gw", BACK_APART["work"]), ("work", BACK_APART["h"]),
    ("work", BACK_APART["gh"]), ("work", BACK_APART["w"]),
])
def test_backward(lib, name, at):  # noqa: F811
    assert norm_back(lib, rows=ROWS, cols=COLS, **{**BACK_APART, name: at}) == 1
    assert "overlaps" in lib.moe_last_error().decode()
