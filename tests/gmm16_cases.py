"""Sizes of the 16-bit products that reach each of the LDS-staged kernel's tiles, with and without items that
blocks share, a block with one item and with several, in whole 16-byte rows and in odd ones.

(form, rows of a tile, shared, rows, groups, n, k), n and k as the calls take them: out is [rows, n] of a
contraction of k (forward, transposed) or [groups, n, k] (weights)."""

FORMS = ["forward", "transposed", "weights"]

# (tile, shared, rows, groups, whole n and k, odd n and k); of a tile's four the first and third give a block one
# item at most, the others more
_PRODUCT = [
    (32, 0, 33, 3, (264, 264), (259, 267)),
    (32, 0, 1537, 40, (1544, 264), (1539, 259)),
    (32, 1, 33, 3, (8, 1544), (9, 1539)),
    (32, 1, 97, 40, (3080, 1544), (3075, 1539)),
    (64, 0, 4096, 3, (136, 264), (131, 259)),
    (64, 0, 2100, 40, (1032, 264), (1027, 259)),
    (64, 1, 97, 1, (1032, 1544), (1027, 1539)),
    (64, 1, 1537, 40, (1544, 1544), (1539, 1539)),
    (128, 0, 3000, 40, (776, 264), (771, 259)),
    (128, 0, 4096, 40, (1032, 264), (1027, 259)),
    (128, 1, 6000, 1, (136, 2056), (131, 2051)),
    (128, 1, 3000, 40, (1544, 1544), (1539, 1539)),
    (160, 0, 6000, 40, (776, 264), (771, 259)),
    (160, 0, 5000, 40, (1032, 264), (1027, 259)),
    (160, 1, 2100, 16, (136, 8200), (131, 8195)),
    (160, 1, 1000, 8, (8200, 2056), (8195, 2051)),
    (192, 0, 3000, 16, (2056, 264), (2051, 259)),
    (192, 0, 3000, 16, (4104, 264), (4099, 259)),
    (192, 1, 161, 1, (8200, 4104), (8195, 4099)),
    (192, 1, 1150, 8, (8200, 2056), (8195, 2051)),
    (256, 0, 1000, 5, (8200, 264), (8195, 259)),
    (256, 0, 3000, 16, (3080, 264), (3075, 259)),
    (256, 1, 1000, 5, (2056, 6152), (2051, 6147)),
    (256, 1, 3000, 16, (4104, 2056), (4099, 2051)),
]
_WEIGHTS = [
    (64, 0, 150, 1, (264, 264), (261, 267)),
    (64, 0, 1000, 8, (4104, 8), (4105, 9)),
    (64, 1, 1537, 1, (8, 72), (9, 73)),
    (64, 1, 5000, 8, (4104, 8), (4105, 9)),
    (128, 0, 300, 3, (6152, 136), (6147, 131)),
    (128, 0, 1000, 8, (72, 8200), (67, 8195)),
    (128, 1, 3000, 1, (4104, 136), (4099, 131)),
    (128, 1, 5000, 8, (72, 8200), (67, 8195)),
    (256, 0, 1000, 8, (4104, 136), (4099, 131)),
    (256, 0, 1000, 8, (6152, 264), (6147, 259)),
    (256, 1, 5000, 1, (8200, 264), (8195, 259)),
    (256, 1, 5000, 8, (8200, 520), (8195, 515)),
]


# (form, tile, rows of each group, groups, n, k): every block has more items than it describes at a time (64)
MANY_ITEMS = [(form, *c) for form in FORMS[:2] for c in [
    (32, 8, 1000, 8200, 8), (64, 3000, 1000, 8, 8), (128, 64, 1000, 4104, 8), (160, 256, 500, 4104, 8),
    (192, 150, 1000, 4104, 8), (256, 30000, 50, 520, 8)]] + [
    ("weights", 64, 8, 500, 8200, 8), ("weights", 128, 8, 500, 2056, 264), ("weights", 256, 8, 500, 4104, 264)]


def offsets(rows, groups):
    """Group offsets near the mean: some rows in front of the first group and behind the last, of four
    groups and more the second empty. None for one group."""
    if groups == 1:
        return None
    ends = [rows * (2 * g + g % 2) // (2 * groups) for g in range(groups + 1)]
    ends[0], ends[-1] = 2, rows - 1
    if groups > 3:
        ends[2] = ends[1]
    return ends


def cases():
    out = []
    for form in FORMS:
        for tile, shared, rows, groups, whole, odd in (_WEIGHTS if form == "weights" else _PRODUCT):
            for n, k in (whole, odd):
                out.append((form, tile, shared, rows, groups, n, k))
    return out
