"""The 16-bit products at the sizes where their kernels change: few rows, tiles of 160 and 192 rows, items shared
between blocks, padded copies of odd sizes, offsets past 32 bits. The bounds are those of test_gpu_gmm16."""
import numpy as np
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say
from oracle import dense
from test_gpu_gmm16 import BF, FP, KINDS, check, f64, on, product, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 24, 25, 31, 32, 33])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 7), (8, 64), (9, 65), (60, 520), (257, 1001), (256, 4096)])
def test_few_rows(rows, n, k):
    """One group: every count around a kernel's 8, 16 and 32 rows, contractions around its steps."""
    kind = (rows + n) % len(KINDS)
    product("forward", rows, 1, n, k, None, kind, seed=rows)
    product("forward", rows, 1, n, k, None, (kind + 1) % len(KINDS), seed=rows, off=1)   # no vectors


@pytest.mark.parametrize("rows", [33, 64, 65, 100, 256, 500, 16384, 16385])
@pytest.mark.parametrize("n,k", [(8, 64), (7, 513), (250, 1000)])
def test_rows_in_several_blocks(rows, n, k):
    """One group of few channels: row blocks of 32, with and without offsets that leave rows outside."""
    if rows > 500 and n > 8:
        return
    kind = rows % len(KINDS)
    product("forward", rows, 1, n, k, None, kind, seed=rows)
    product("forward", rows, 1, n, k, [0, rows], kind, seed=rows)
    product("forward", rows, 1, n, k, [5, rows - 6], kind, seed=rows, off=1)


def test_one_group_needs_one_workspace():
    """The workspace that is asked for without offsets is the one a call of one group with offsets takes."""
    for rows, n, k in ((64, 256, 7168), (600, 256, 7168), (600, 256, 7169), (40, 4096, 512)):
        x, w = on(values((rows, k), BF, 0)), on(values((1, n, k), BF, 1))
        o = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        need = rp._sized("moe_grouped_matmul_workspace_size", rows, 1, n, k, 0)
        ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device=DEV)
        say(f"one group {rows} {n} {k}: {need} bytes")
        assert torch.equal(rp.grouped_matmul(x, w, o, workspace=ws), rp.grouped_matmul(x, w, workspace=ws))


def ragged(rows, groups, seed):
    rng = np.random.default_rng(seed)
    return [0, *np.sort(rng.integers(0, rows + 1, groups - 1)).tolist(), rows]


FEW = {
    "one each": [0, 1, 2, 3, 4, 5, 6, 7, 8],
    "gaps": [0, 0, 0, 3, 3, 4, 4, 13, 13],
    "all in the last": [0, 0, 0, 0, 0, 0, 0, 0, 16],
    "all in the first": [0, 32, 32, 32, 32, 32, 32, 32, 32],
    "rows outside": [2, 5, 5, 9, 12, 12, 20, 21, 27],
    "none": [0] * 9,
}


@pytest.mark.parametrize("name", list(FEW))
@pytest.mark.parametrize("n,k", [(8, 64), (61, 100), (264, 1000)])
def test_few_rows_of_groups(name, n, k):
    off = FEW[name]
    rows = off[-1] + (3 if name == "rows outside" else 0) or 4
    for kind in range(4):
        product("forward", rows, 8, n, k, off, kind, seed=kind)
    product("forward", rows, 8, n, k, off, 0, off=5)


@pytest.mark.parametrize("rows,groups,n,k", [(8, 1, 16400, 64), (8, 12, 1200, 504), (12, 12, 1200, 2040), (16, 12, 1200, 2056),
                                             (16, 3, 1203, 72), (30, 30, 300, 504), (32, 30, 520, 520), (32, 1, 4200, 72)])
def test_few_rows_of_many_channels(rows, groups, n, k):
    """Around the sizes where tiles take over from the kernel of few rows, aligned and not."""
    off = None if groups == 1 else ragged(rows, groups, n)
    for kind in (0, 1):
        product("forward", rows, groups, n, k, off, kind)
    product("forward", rows, groups, n, k, off, 2, off=3)


def test_few_rows_of_many_groups():
    """The most groups, and groups past one wave's count of them."""
    for groups in (63, 64, 65, 130, 1024):
        off = [0] * (groups // 2) + [1] * (groups // 4) + [5] * (groups - groups // 2 - groups // 4) + [9]
        product("forward", 9, groups, 24, 72, off, groups % 4)


def test_few_rows_bad_offsets_and_bad_neighbours():
    """Offsets past the rows are cut there. What a group does not own does not reach its rows: neighbours'
    infinities, and those of the channels and the rows behind it."""
    x, w = values((12, 72), BF, 0), values((3, 20, 72), BF, 1)
    want, mag = dense.grouped_matmul(f64(x), f64(w), [0, 0, 5, 12])
    got = rp.grouped_matmul(on(x), on(w), torch.tensor([-7, -2, 5, 900], dtype=torch.int32, device=DEV))
    check(got, want, mag, 72, BF)
    o = torch.tensor([0, 4, 7, 12], dtype=torch.int32, device=DEV)
    clean = rp.grouped_matmul(on(x), on(w), o)
    xs, ws = on(x), on(w)
    xs[4:7] = float("nan")
    ws[1] = float("inf")
    ws[2, 7] = float("nan")
    got = rp.grouped_matmul(xs, ws, o)
    assert torch.equal(got[:4], clean[:4]) and bool(got[4:7].isnan().all())
    keep = torch.arange(20) != 7
    assert torch.equal(got[7:, keep], clean[7:, keep]) and bool(got[7:, 7].isnan().all())


@pytest.mark.parametrize("form", ["forward", "transposed"])
@pytest.mark.parametrize("mean", [100, 150, 180, 240, 300])
def test_rows_of_a_group(form, mean):
    """Groups whose rows fill one tile of 128, 160, 192, 256 rows and two of 160, and ragged ones of that mean."""
    for groups in (1, 40):
        rows = mean * groups
        even = None if groups == 1 else [mean * g for g in range(groups + 1)]
        product(form, rows, groups, 520, 648, even, 0)
        if groups > 1:
            product(form, rows, groups, 264, 136, ragged(rows, groups, mean), 1)


@pytest.mark.parametrize("form,rows,groups,n,k", [
    ("forward", 300, 1, 520, 7168), ("forward", 700, 3, 264, 4104), ("transposed", 300, 1, 4096, 520),
    ("transposed", 900, 4, 4104, 264), ("weights", 4100, 1, 130, 300), ("weights", 9000, 3, 72, 264),
    ("weights", 8192, 1, 256, 1032)])
def test_shared_items(form, rows, groups, n, k):
    """Few tiles of a long contraction: several blocks share one and join their sums."""
    off = None if groups == 1 else [0, *[rows * g // groups + 5 for g in range(1, groups)], rows]
    for kind in (1, 2):
        product(form, rows, groups, n, k, off, kind)


@pytest.mark.parametrize("form", ["forward", "transposed", "weights"])
@pytest.mark.parametrize("n,k", [(61, 2051), (2049, 100), (515, 517), (8, 3)])
def test_padded_copies(form, n, k):
    """Odd contractions and widths of more rows than the kernel of few takes."""
    product(form, 333, 1, n, k, None, 0)
    product(form, 2500, 3, n, k, [0, 700, 700, 2500], 1)


def test_workspace_of_the_caller():
    """A workspace of the size asked for, full of NaN, gives the same bits as the library's own; a smaller one is not
    used."""
    for form, rows, n, k in (("forward", 300, 520, 7168), ("transposed", 333, 2049, 515), ("weights", 4100, 130, 301)):
        say(f"workspace {form} {rows} {n} {k}")
        x, w, g = on(values((rows, k), BF, 0)), on(values((1, n, k), BF, 1)), on(values((rows, n), BF, 2))

        def call(ws=None):
            if form == "weights":
                return rp.grouped_matmul_wgrad(g, x, workspace=ws)
            return rp.grouped_matmul(x if form == "forward" else g, w, transpose_w=form == "transposed", workspace=ws)

        want = call()
        if form == "weights":
            need = rp._sized("moe_grouped_matmul_wgrad_workspace_size", rows, 1, n, k)
        else:
            need = rp._sized("moe_grouped_matmul_workspace_size", rows, 1, n, k, int(form == "transposed"))
        assert need > 0
        ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)   # (NaN as 16 and as 32 bits)
        for _ in range(2):
            assert torch.equal(call(ws), want)
        small = torch.full((16,), 255, dtype=torch.uint8, device=DEV)
        assert torch.equal(call(small), want) and bool((small == 255).all())


def test_graphs_that_share_a_workspace():
    """Two graphs with one workspace, replayed in turn on one stream."""
    n, k, rows = 515, 4099, 333
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    x, w, g = on(values((rows, k), BF, 0)), on(values((1, n, k), BF, 1)), on(values((rows, n), BF, 2))

    def first():
        return rp.grouped_matmul(x, w, workspace=ws)

    def second():
        return rp.grouped_matmul(g, w, transpose_w=True, workspace=ws), rp.grouped_matmul_wgrad(g, x, workspace=ws)

    first(), second()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in (first, second):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f())
    for seed in range(3):
        x.copy_(values((rows, k), BF, 50 + seed))
        g.copy_(values((rows, n), BF, 60 + seed))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        a, (b, c) = first(), second()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], a) and torch.equal(outs[1][0], b) and torch.equal(outs[1][1], c)


def exact_rows(x, w):
    """Rows x (bf16) by w [n, k] in 64 bits, and the sums of magnitudes."""
    a, b = f64(x), f64(w)
    return a @ b.T, np.abs(a) @ np.abs(b).T


@pytest.mark.parametrize("rows,groups,n,k", [(40, 17, 16384, 8200), (20, 17, 16384, 8200), (300, 9, 16384, 16392)])
def test_weights_past_32_bits(rows, groups, n, k):
    """Weights of more than 2^31 elements: the rows of the last group, and of the first."""
    say(f"weights past 32 bits: {rows} rows, {groups} x {n} x {k}")
    gen = torch.Generator(device=DEV).manual_seed(0)
    w = torch.empty((groups, n, k), dtype=BF, device=DEV)
    for g in range(groups):
        w[g].normal_(0, k ** -0.5, generator=gen)
    x, y = (torch.randn((rows, c), generator=gen, device=DEV).to(BF) for c in (k, n))
    o = torch.tensor([0, rows // 2, *[rows // 2] * (groups - 2), rows], dtype=torch.int32, device=DEV)
    got, back = rp.grouped_matmul(x, w, o), rp.grouped_matmul(y, w, o, transpose_w=True)
    for g, r in ((0, 0), (0, rows // 2 - 1), (groups - 1, rows // 2), (groups - 1, rows - 1)):
        want, mag = exact_rows(x[r:r + 1], w[g, -64:])
        check(got[r:r + 1, -64:], want, mag, k, BF)
        want, mag = exact_rows(y[r:r + 1], w[g, :, -64:].T)
        check(back[r:r + 1, -64:], want, mag, n, BF)


def test_rows_past_32_bits():
    """Rows of more than 2^31 elements, and outputs; the gradient by weights of more than 2^31 elements."""
    rows, k, n = 270000, 8200, 40
    say(f"rows past 32 bits: {rows} x {k}")
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.empty((rows, k), dtype=BF, device=DEV).normal_(0, 1, generator=gen)
    w = torch.randn((1, n, k), generator=gen, device=DEV).mul_(k ** -0.5).to(BF)
    got = rp.grouped_matmul(x, w)
    for r in (0, 131071, 262143, rows - 1):
        want, mag = exact_rows(x[r:r + 1], w[0])
        check(got[r:r + 1], want, mag, k, BF)
    back = rp.grouped_matmul(got, w, transpose_w=True)
    for r in (0, 262143, rows - 1):
        want, mag = exact_rows(got[r:r + 1], w[0].T)
        check(back[r:r + 1], want, mag, n, BF)
    del back
    o = torch.tensor([0, 100, rows - 200, rows], dtype=torch.int32, device=DEV)
    gw = rp.grouped_matmul_wgrad(got, x, o, out_dtype=FP)
    want, mag = exact_rows(got[-200:, :8].T, x[-200:, -64:].T)
    check(gw[2, :8, -64:], want, mag, 200, FP)
    del gw, x
    groups, n, k, rows = 17, 16384, 8200, 70
    say(f"gradient past 32 bits: {groups} x {n} x {k}")
    a, b = (torch.randn((rows, c), generator=gen, device=DEV).to(BF) for c in (n, k))
    o = torch.tensor([0, 30, *[30] * (groups - 2), rows], dtype=torch.int32, device=DEV)
    gw = rp.grouped_matmul_wgrad(a, b, o)
    assert not bool(gw[1:-1].any())
    for g, lo, hi in ((0, 0, 30), (groups - 1, 30, rows)):
        want, mag = exact_rows(a[lo:hi, -64:].T, b[lo:hi, -64:].T)
        check(gw[g, -64:, -64:], want, mag, hi - lo, BF)
