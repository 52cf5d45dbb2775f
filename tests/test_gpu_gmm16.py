"""The 16-bit products of expert groups on the GPU against float64: forward, transposed (the
gradient by the input) and the gradient by the weights.

Bound: products of 16-bit values are exact in fp32. An MFMA adds at least 16 of them to the
accumulator; allowing it one unit 2^-23 of the sum of the magnitudes, and 64 more units where parts
of a long sum are joined: (L / 16 + 64) 2^-23 sum |a| |b| for a sum of L products; then the rounding to
the output's type, eps / 2 relative and half its smallest subnormal (fp32: none)."""
import numpy as np
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say
from oracle import dense

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
KINDS = [(BF, BF), (HF, FP), (BF, FP), (HF, HF)]
FORMS = ["forward", "transposed", "weights"]


def values(shape, dtype, seed, std=1.0, spread=2.0):
    gen = torch.Generator().manual_seed(seed)
    scale = torch.exp(torch.rand((*shape[:-1], 1), generator=gen) * 2 * spread - spread) * std
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def on(t, off=0):
    """t on the GPU, `off` elements behind a 16-byte boundary."""
    buf = torch.empty((t.numel() + 8,), dtype=t.dtype, device=DEV)
    out = buf[off:off + t.numel()].view(t.shape)
    out.copy_(t)
    return out


def check(got, want, mag, length, out_dtype, where=""):
    err = (length / 16 + 64) * 2.0 ** -23 * mag
    f = torch.finfo(out_dtype)
    e, t = (0.0, 0.0) if out_dtype == FP else (f.eps / 2, f.smallest_normal * f.eps / 2)
    bound = err + e * (np.abs(want) + err) + t + 2.0 ** -120
    excess = np.abs(f64(got) - want) / bound
    assert np.all(excess <= 1.0), (where, float(np.nanmax(excess)), np.argwhere(~(excess <= 1.0))[:4].tolist())


def product(form, rows, groups, n, k, offsets=None, kind=0, seed=0, off=0):
    """One call of a form in the sizes of the forward product [rows, k] x [n, k], checked; what it was given and made."""
    dtype, out_dtype = KINDS[kind]
    say(f"{form} rows={rows} groups={groups} n={n} k={k} {dtype} -> {out_dtype} offset={off} "
        f"offsets={None if offsets is None else list(offsets)[:8]}")
    o = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    if form == "weights":
        g, x = values((rows, n), dtype, seed), values((rows, k), dtype, seed + 1)
        shape = (n, k) if offsets is None else (groups, n, k)
        out = torch.full(shape, 7.0, dtype=out_dtype, device=DEV)
        got = rp.grouped_matmul_wgrad(on(g, off), on(x, off), o, out=out)
        assert got is out
        want, mag = dense.grouped_matmul_wgrad(f64(g), f64(x), offsets)
        for i, (lo, hi) in enumerate(dense.groups(offsets, rows)):
            check(got.view(groups, n, k)[i], want[i], mag[i], hi - lo, out_dtype, i)
        return (g, x), got
    trans = form == "transposed"
    con, width = (n, k) if trans else (k, n)
    x, w = values((rows, con), dtype, seed), values((groups, n, k), dtype, seed + 1, k ** -0.5)
    out = torch.full((rows, width), 7.0, dtype=out_dtype, device=DEV)
    wd = on(w, off)
    got = rp.grouped_matmul(on(x, off), wd[0] if offsets is None else wd, o, transpose_w=trans, out=out)
    assert got is out
    want, mag = dense.grouped_matmul(f64(x), f64(w), offsets, trans)
    inside = ~np.isnan(want[:, 0]) if rows else np.zeros(0, bool)
    check(got[torch.from_numpy(inside).to(DEV)], want[inside], mag[inside], con, out_dtype)
    assert bool((got[torch.from_numpy(~inside).to(DEV)] == 7).all())   # left as they were
    return (x, w), got


SIZES = [(1, 1, 1), (1, 16, 128), (1, 256, 7168), (2, 48, 384), (3, 60, 1000), (15, 130, 72), (16, 64, 512),
         (17, 1000, 640), (33, 272, 1152), (64, 256, 2048), (100, 61, 33), (129, 1296, 264), (255, 320, 904),
         (257, 264, 520), (300, 2056, 1024), (520, 776, 8), (700, 512, 7168), (1100, 8, 264), (40, 7, 4100)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_dense(form, rows, n, k):
    for kind in range(len(KINDS)):
        product(form, rows, 1, n, k, None, kind, seed=rows + kind)


GROUPED = {
    "one row each": [0, 1, 2, 3, 4, 5, 6],
    "empty ends": [0, 0, 40, 40, 41, 60, 60],
    "tile ends": [0, 16, 48, 112, 240, 496, 497],
    "one holds all": [0, 0, 0, 600, 600, 600, 600],
    "ragged": [0, 3, 131, 131, 390, 437, 777],
    "none": [0, 0, 0, 0, 0, 0, 0],
    "rows outside": [5, 5, 9, 150, 151, 160, 161],
    "large": [0, 300, 900, 1164, 1164, 1420, 2200],
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("name", list(GROUPED))
@pytest.mark.parametrize("n,k", [(64, 256), (328, 1416), (61, 100), (1032, 520)])
def test_grouped(form, name, n, k):
    off = GROUPED[name]
    rows = off[-1] + (4 if name == "rows outside" else 0) or 3
    for kind in range(2 if rows > 1000 else 4):
        product(form, rows, 6, n, k, off, kind, seed=kind)


@pytest.mark.parametrize("form", FORMS)
def test_many_groups(form):
    """More groups than rows, hundreds of groups of a few rows, and the most groups."""
    rng = np.random.default_rng(0)
    for rows, groups, n, k in [(5, 300, 64, 128), (900, 200, 64, 136), (3000, 1024, 40, 64)]:
        off = [0, *np.sort(rng.integers(0, rows + 1, groups - 1)).tolist(), rows]
        product(form, rows, groups, n, k, off, 2)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k", [(64, 256), (264, 1000)])
def test_unaligned(form, n, k):
    """Tensors that start at an odd element: the kernel for every shape."""
    product(form, 77, 1, n, k, None, 0, off=3)
    product(form, 130, 3, n, k, [2, 50, 50, 129], 1, off=1)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k", [(72, 200), (264, 1000), (61, 33), (520, 64)])
def test_what_belongs_to_others_is_not_touched(form, n, k):
    """Infinities and NaN in rows outside the groups, and in every second group, leave the other groups' results as they
    are without them, bit for bit: nothing of a neighbour is multiplied by zero."""
    off, rows = [3, 40, 41, 170, 300, 301, 420], 430
    dtype = BF
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    spoiled = torch.ones(rows, dtype=torch.bool)
    for g in (0, 2, 4):
        spoiled[off[g]:off[g + 1]] = False

    def with_bad(t):
        t = t.clone()
        t[spoiled] = float("nan")
        t[spoiled, ::3] = float("inf")
        return t

    if form == "weights":
        g, x = values((rows, n), dtype, 0), values((rows, k), dtype, 1)
        clean, bad = (rp.grouped_matmul_wgrad(on(a), on(b), o) for a, b in ((g, x), (with_bad(g), with_bad(x))))
        assert torch.equal(clean[0::2], bad[0::2])
        return
    trans = form == "transposed"
    x, w = values((rows, n if trans else k), dtype, 0), values((6, n, k), dtype, 1)
    wb = w.clone()
    wb[1::2] = float("nan")
    clean, bad = (rp.grouped_matmul(on(a), on(b), o, transpose_w=trans) for a, b in ((x, w), (with_bad(x), wb)))
    for g in (0, 2, 4):
        assert torch.equal(clean[off[g]:off[g + 1]], bad[off[g]:off[g + 1]])


@pytest.mark.parametrize("n,k", [(72, 200), (264, 1000)])
def test_a_bad_row_or_channel_stays_in_its_own(n, k):
    """NaN in one row of x spoils that row of out, in one channel of w that column, and nothing else."""
    rows = 300
    x, w = values((rows, k), BF, 0), values((n, k), BF, 1)
    clean = rp.grouped_matmul(on(x), on(w))
    x[100], w[5, k - 1] = float("nan"), float("inf")
    bad = rp.grouped_matmul(on(x), on(w))
    keep_r, keep_c = torch.arange(rows, device=DEV) != 100, torch.arange(n, device=DEV) != 5
    assert torch.equal(bad[keep_r][:, keep_c], clean[keep_r][:, keep_c])
    assert bool(bad[100].isnan().all()) and not bool(bad[:, 5].isfinite().any())


def test_offsets_outside_the_rows():
    """Offsets that run past the rows are cut there; nothing behind is read or written."""
    x, w = values((50, 64), BF, 0), values((2, 32, 64), BF, 1)
    o = torch.tensor([-5, 20, 900], dtype=torch.int32, device=DEV)
    got = rp.grouped_matmul(on(x), on(w), o)
    want, mag = dense.grouped_matmul(f64(x), f64(w), [0, 20, 50])
    check(got, want, mag, 64, BF)
    g = values((50, 32), BF, 2)
    got = rp.grouped_matmul_wgrad(on(g), on(x), o)
    want, mag = dense.grouped_matmul_wgrad(f64(g), f64(x), [0, 20, 50])
    check(got, want, mag, 50, BF)


def test_no_rows():
    x, w, g = (torch.zeros(s, dtype=BF, device=DEV) for s in ((0, 64), (3, 32, 64), (0, 32)))
    o = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert rp.grouped_matmul(x, w, o).shape == (0, 32)
    assert rp.grouped_matmul(g, w, o, transpose_w=True).shape == (0, 64)
    gw = rp.grouped_matmul_wgrad(g, x, o, out=torch.full((3, 32, 64), 7.0, device=DEV))
    assert not gw.any()
    assert not rp.grouped_matmul_wgrad(g, x).any()


def test_captured_replayed_and_two_streams():
    off = [0, 100, 100, 350, 700]
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    n, k, rows = 264, 1024, 700
    x, w, g = on(values((rows, k), BF, 0)), on(values((4, n, k), BF, 1)), on(values((rows, n), BF, 2))

    def step(x, w, g):
        return (rp.grouped_matmul(x, w, o), rp.grouped_matmul(g, w, o, transpose_w=True),
                rp.grouped_matmul_wgrad(g, x, o, out_dtype=FP), rp.grouped_matmul(x[:2], w[0]),
                rp.grouped_matmul_wgrad(g, x))

    step(x, w, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, w, g)
    for seed in range(3):
        for t, i in ((x, 0), (w, 1), (g, 2)):
            t.copy_(values(tuple(t.shape), BF, 10 * seed + i))
        graph.replay()
        want = step(x.clone(), w.clone(), g.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([step(x, w, g) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for runs in got for run in runs for a, b in zip(run, want))


def test_gradients_against_differences():
    """The loss sum(out q) is bilinear: differences along a direction of size 1 give its gradient but
    for the roundings, (L / 16 + 64) 2^-23 of the magnitudes in each product (fp32 out)."""
    off, rows, n, k = [0, 33, 33, 90], 90, 40, 72
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    x, w, q = values((rows, k), BF, 0, spread=0.5), values((3, n, k), BF, 1, spread=0.5), values((rows, n), BF, 2, spread=0.5)
    gx = rp.grouped_matmul(on(q), on(w), o, transpose_w=True, out_dtype=FP)
    gw = rp.grouped_matmul_wgrad(on(q), on(x), o, out_dtype=FP)

    def loss(x, w):
        return float((f64(rp.grouped_matmul(on(x), on(w), o, out_dtype=FP)) * f64(q)).sum())

    for seed in range(3):
        # directions on the grid of the values, so that x +- vx is exact in bf16: signs, at most one step of x
        vx = torch.sign(values(tuple(x.shape), FP, 30 + seed)).to(BF) * 0
        vx[seed::7] = x[seed::7]          # x itself along some rows: 2 x and 0
        vw = torch.zeros_like(w)
        vw[:, seed::5] = w[:, seed::5]
        mag = float((dense.grouped_matmul(np.abs(f64(x)) * 2, np.abs(f64(w)) * 2, off)[1] * np.abs(f64(q))).sum())
        for a, b, got in (((x + vx, w), (x - vx, w), (f64(gx) * f64(vx)).sum()), ((x, w + vw), (x, w - vw), (f64(gw) * f64(vw)).sum())):
            assert abs((loss(*a) - loss(*b)) / 2 - got) <= 2 * (90 / 16 + 64) * 2.0 ** -23 * mag
