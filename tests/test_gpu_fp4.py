"""The MXFP4 product on the GPU against the float64 oracle: x as codes or quantised in the
call, grouped and dense, ND and packed weights, odd and ragged sizes.

Bound: the FP4 products are exact, a K step of 128 adds its products and the accumulator in
fp32; a wave's partial sums (up to 8) are added in fp32. Allowing one unit 2^-23 of the sum
of the products' magnitudes per K step and per partial sum: (K / 128 + 8) 2^-23 sum |x| |w|;
then the rounding to the output type, eps / 2 relative."""
import ctypes

import numpy as np
import pytest
import torch

import moe_inputs
import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say, to_dev
from oracle import mxfp

pytestmark = pytest.mark.gpu


def fp4(v):
    """(packed codes, scales, dequantised float64) of v by the oracle."""
    c, s = mxfp.quantize(v, "e2m1")
    return mxfp.pack_fp4(c), s, mxfp.dequantize(c, s, "e2m1")


def operands(rows, groups, n, k, seed=0, dtype=None, spread=2.0):
    """x (codes, scales or values), its float64 value, and w codes, scales, float64 value."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * np.exp(rng.uniform(-spread, spread, (rows, 1)))
    if dtype is not None:
        t = torch.from_numpy(x.astype(np.float32)).to(dtype)
        x = t.double().numpy()
    w = rng.standard_normal((groups, n, k)) / np.sqrt(k)
    wc, ws, wv = fp4(w)
    xc, xs, xv = fp4(x) if rows else (np.zeros((0, k // 2), np.uint8), np.zeros((0, k // 32), np.uint8), x)
    return (t if dtype is not None else (xc, xs)), xv, wc, ws, wv


def check(got, x, w, offsets, out_dtype):
    got = got.cpu().double().numpy()
    k = x.shape[1]
    for g, (lo, hi) in enumerate(zip(offsets[:-1], offsets[1:])):
        if hi <= lo:
            continue
        want, mag = x[lo:hi] @ w[g].T, np.abs(x[lo:hi]) @ np.abs(w[g]).T
        err = (k / 128 + 8) * 2.0 ** -23 * mag
        bound = err + torch.finfo(out_dtype).eps / 2 * (np.abs(want) + err) + 2.0 ** -120
        excess = np.abs(got[lo:hi] - want) / bound
        assert np.all(excess <= 1.0), (g, float(excess.max()))


def product(rows, groups, n, k, offsets=None, dtype=None, out_dtype=torch.bfloat16, packed=False, seed=0):
    say(f"mxfp4_matmul rows={rows} groups={groups} n={n} k={k} x={dtype} out={out_dtype} packed={packed} "
        f"offsets={None if offsets is None else list(offsets)[:8]}")
    x, xv, wc, ws, wv = operands(rows, groups, n, k, seed, dtype)
    w, s = to_dev(wc), to_dev(ws)
    if packed:
        w, s = rp.pack_weights(w, s, fp4=True)
    kw = dict(x_scales=to_dev(x[1])) if dtype is None else {}
    xd = to_dev(x[0]) if dtype is None else x.to(DEV)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    out = torch.full((rows, n), 7.0, dtype=out_dtype, device=DEV)
    got = rp.mxfp4_matmul(xd, w, s, group_offsets=off, out=out,
                          weight_format=rp.WEIGHTS_PACKED if packed else rp.WEIGHTS_ND, **kw)
    assert got is out
    torch.cuda.synchronize()
    offsets = [0, rows] if offsets is None else offsets
    check(got, xv, wv, offsets, out_dtype)
    assert bool((got[:offsets[0]] == 7).all()) and bool((got[offsets[-1]:] == 7).all())   # left as they were
    return xd, w, s, got


KINDS = [(None, torch.bfloat16, False), (torch.bfloat16, torch.bfloat16, True), (torch.float16, torch.float32, False),
         (torch.float32, torch.bfloat16, False), (None, torch.float32, True)]


@pytest.mark.parametrize("rows,n,k", [(1, 16, 128), (1, 2048, 1408), (2, 48, 384), (15, 1040, 256), (16, 64, 512),
                                      (17, 4096, 640), (33, 272, 1152), (64, 256, 2048), (100, 528, 768),
                                      (129, 1296, 256), (257, 320, 896), (300, 2064, 1024), (700, 512, 7168)])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_dense(rows, n, k, kind):
    dtype, out_dtype, packed = KINDS[kind]
    product(rows, 1, n, k, None, dtype, out_dtype, packed, seed=rows)


GROUPED = {
    "one row each": [0, 1, 2, 3, 4, 5, 6],
    "empty ends": [0, 0, 40, 40, 41, 60, 60],
    "tile ends": [0, 16, 48, 112, 240, 496, 497],
    "one holds all": [0, 0, 0, 600, 600, 600, 600],
    "ragged": [0, 3, 131, 131, 390, 437, 777],
    "none": [0, 0, 0, 0, 0, 0, 0],
    "rows outside": [5, 5, 9, 150, 151, 160, 161],
}


@pytest.mark.parametrize("name", list(GROUPED))
@pytest.mark.parametrize("n,k", [(64, 256), (336, 1408), (2048, 512)])
def test_grouped(name, n, k):
    off = GROUPED[name]
    for i, (dtype, out_dtype, packed) in enumerate(KINDS):
        product(off[-1] + (4 if name == "rows outside" else 0) or 3, 6, n, k, off, dtype, out_dtype, packed, seed=i)


def test_many_groups():
    """More groups than rows, and hundreds of groups of a few rows."""
    rng = np.random.default_rng(0)
    for rows, groups in [(5, 300), (900, 200)]:
        off = [0, *np.sort(rng.integers(0, rows + 1, groups - 1)).tolist(), rows]
        product(rows, groups, 64, 128, off, torch.bfloat16, torch.float32, False)
        product(rows, groups, 64, 128, off, None, torch.bfloat16, True)


@pytest.mark.parametrize("rows", [3, 600])
def test_quantisation_of_every_bf16_value(rows):
    """x against an identity weight (code 2 = 1.0 on the diagonal, scale 2^0): the output is
    DQ(Q_MX(x)) itself, exact but for fp32's subnormal range. Every finite bf16 value, in random
    groups and in groups of neighbouring magnitudes, by the kernel for few rows and for many."""
    bits = np.arange(65536, dtype=np.uint32)
    bits = bits[np.isfinite((bits << 16).view(np.float32))].astype(np.uint16)
    k = 256
    w = np.zeros((1, k, k), dtype=np.uint8)
    w[0, np.arange(k), np.arange(k)] = 2
    wc, ws = to_dev(mxfp.pack_fp4(w)), torch.full((1, k, k // 32), 127, dtype=torch.uint8, device=DEV)
    for order in ("random", "sorted"):
        b = np.random.default_rng(1).permutation(bits)
        if order == "sorted":
            b = bits[np.argsort(np.abs(mxfp.bf16_from_bits(bits)), kind="stable")]
        b = np.concatenate([b, np.zeros((-b.size) % k, np.uint16)]).reshape(-1, k)
        c, s = mxfp.quantize(mxfp.bf16_from_bits(b), "e2m1")
        want = mxfp.dequantize(c, s, "e2m1")
        x = torch.from_numpy(b.astype(np.int16)).view(torch.bfloat16).to(DEV)
        for dtype in (torch.bfloat16, torch.float32):
            say(f"mxfp4_matmul every bf16 value rows={rows} {order} {dtype}")
            for lo in range(0, x.shape[0], rows):
                part = x[lo:lo + rows].to(dtype)
                part = torch.cat([part, part.new_ones((rows - part.shape[0], k))])
                got = rp.mxfp4_matmul(part, wc, ws, out_dtype=torch.float32).cpu().double().numpy()
                ref = want[lo:lo + rows]
                got = got[:ref.shape[0]]
                normal = np.abs(ref) >= 2.0 ** -126
                assert np.array_equal(got[normal], ref[normal])
                assert np.all(np.abs(got[~normal]) <= 2.0 ** -126)


def test_same_result_as_codes():
    """x quantised in the call gives the bits of the product of mx_quantize's codes; repeated
    calls give the same bits."""
    for rows, n, k in [(1, 512, 1024), (37, 512, 1408), (520, 768, 640)]:
        x = torch.randn((rows, k), generator=torch.Generator().manual_seed(rows)).to(torch.bfloat16).to(DEV)
        wc, ws, _ = fp4(np.random.default_rng(0).standard_normal((1, n, k)))
        w, s = to_dev(wc), to_dev(ws)
        codes, scales = rp.mx_quantize(x, rp.QUANT_MXFP4)
        a = rp.mxfp4_matmul(x, w[0], s[0], out_dtype=torch.float32)
        b = rp.mxfp4_matmul(codes, w, s, x_scales=scales, out_dtype=torch.float32)
        assert torch.equal(a, b) and torch.equal(a, rp.mxfp4_matmul(x, w, s, out_dtype=torch.float32))


def test_no_rows_and_given_workspace():
    w = torch.zeros((2, 32, 64), dtype=torch.uint8, device=DEV)
    s = torch.zeros((2, 32, 4), dtype=torch.uint8, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    got = rp.mxfp4_matmul(torch.empty((0, 128), device=DEV, dtype=torch.bfloat16), w, s, group_offsets=off)
    assert tuple(got.shape) == (0, 32)
    x = torch.randn((300, 128), device=DEV)
    off = torch.tensor([0, 150, 300], dtype=torch.int32, device=DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    a = rp.mxfp4_matmul(x, w, s, group_offsets=off, workspace=ws)
    assert torch.equal(a, rp.mxfp4_matmul(x, w, s, group_offsets=off))


def test_captured_and_replayed_on_two_streams():
    """Two captured graphs of different sizes, replayed in turn on changed inputs with eager
    work between, and an eager call on another stream."""
    held = []
    for rows, dtype in [(8, torch.bfloat16), (700, torch.float32)]:
        wc, ws, _ = fp4(np.random.default_rng(rows).standard_normal((3, 272, 640)))
        w, s = to_dev(wc), to_dev(ws)
        off = torch.tensor([0, rows // 4, rows // 4, rows], dtype=torch.int32, device=DEV)
        x = torch.randn((rows, 640), device=DEV).to(dtype)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            first = rp.mxfp4_matmul(x, w, s, group_offsets=off)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(first, rp.mxfp4_matmul(x, w, s, group_offsets=off))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rp.mxfp4_matmul(x, w, s, group_offsets=off)
        held.append((graph, x, w, s, off, out))
    for _ in range(4):
        for graph, x, *_ in held:
            x.copy_(torch.randn_like(x))
            graph.replay()
        torch.cuda.synchronize()
        for graph, x, w, s, off, out in held:
            assert torch.equal(out, rp.mxfp4_matmul(x, w, s, group_offsets=off))


def test_router_to_expert_product():
    """Logits -> gate_topk -> init_routing (MXFP4 rows) -> mxfp4_matmul over the active experts,
    without a step between but the offsets: against the oracle of the same chain."""
    n, e, k, h, width = 150, 16, 4, 256, 96
    first, last = 4, 12
    cfg = moe_inputs.config("tiny", tokens=n, hidden=h, experts=e, topk=k)
    x = moe_inputs.activations(cfg)
    logits = torch.randn((n, e), generator=torch.Generator().manual_seed(2))
    wc, ws, wv = fp4(np.random.default_rng(5).standard_normal((last - first, width, h)))
    ids, _ = rp.gate_topk(logits.to(DEV), k)
    rows, _, ends, scales, avail = rp.init_routing(x.to(DEV), ids, e, (first, last), rp.QUANT_MXFP4,
                                                   expert_tokens_num_type=0)
    off = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
    out = torch.full((n * k, width), 3.0, device=DEV)
    rp.mxfp4_matmul(rows, to_dev(wc), to_dev(ws), x_scales=scales, group_offsets=off, out=out)
    flat = ids.cpu().numpy().reshape(-1)
    order = np.argsort(flat, kind="stable")
    order = order[(flat[order] >= first) & (flat[order] < last)]
    assert int(avail) == order.size
    xv = fp4(x.double().numpy())[2][order // k]
    bounds = [int(v) for v in off.cpu()]
    check(out[:order.size], xv, wv, bounds, torch.float32)
    assert bool((out[order.size:] == 3).all())


def test_more_items_than_a_block_lists_at_once():
    """A product of so many tiles that every block of the many-rows kernel computes over 256
    (it describes 64 at a time): rows from all over it against the oracle."""
    rows, n, k = 300_000, 16384, 128
    say(f"mxfp4_matmul rows={rows} n={n} k={k}")
    rng = np.random.default_rng(0)
    x, xv, wc, ws, wv = operands(4096, 1, n, k, seed=1)
    pick = torch.from_numpy(rng.integers(0, 4096, rows))   # rows of x, many times over
    codes, scales = to_dev(x[0])[pick.to(DEV)], to_dev(x[1])[pick.to(DEV)]
    got = rp.mxfp4_matmul(codes, to_dev(wc), to_dev(ws), x_scales=scales)
    some = np.sort(rng.choice(rows, 700, replace=False))
    some[0], some[-1] = 0, rows - 1
    check(got[torch.from_numpy(some).to(DEV)], xv[pick.numpy()[some]], wv, [0, some.size], torch.bfloat16)
    # every row that repeats a row of x repeats its result
    first = torch.zeros(4096, dtype=torch.int64, device=DEV)
    first[pick.flip(0).to(DEV)] = torch.arange(rows - 1, -1, -1, device=DEV)
    for lo in range(0, rows, 50_000):
        part = pick[lo:lo + 50_000].to(DEV)
        assert torch.equal(got[lo:lo + 50_000], got[first[part]])


def drawn(groups, n, k, seed):
    """Random weight codes and scales with their float64 value, made without quantising."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (groups, n, k // 2), dtype=np.uint8)
    s = rng.integers(118, 128, (groups, n, k // 32), dtype=np.uint8)
    table = mxfp.dequantize(np.arange(16, dtype=np.uint8).repeat(32).reshape(16, 32), np.full((16, 1), 127, np.uint8),
                            "e2m1")[:, 0]
    v = np.stack([table[c & 15], table[c >> 4]], axis=-1).reshape(groups, n, k)
    v *= np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=-1)
    return c, s, v


def scattered(rows, groups, rng, outside):
    """Offsets of groups of unequal sizes, some without rows, `outside` rows before and behind."""
    share = rng.gamma(1.5, size=groups) * (rng.random(groups) > 0.15)
    sizes = rng.multinomial(rows - 2 * outside, share / share.sum())
    return [outside, *(outside + np.cumsum(sizes)).tolist()]


@pytest.mark.parametrize("groups,per,n,k", [
    (90, 1, 2064, 128), (90, 9, 2064, 128), (80, 3, 1136, 640), (80, 18, 1136, 640), (300, 1, 528, 512),   # one small tile
    (40, 30, 1136, 640), (60, 45, 1040, 384),                                                             # a tile of 64
    (3, 234, 1040, 896), (5, 156, 2000, 1408),                                       # tiles of 64, to occupy the chip
    (30, 100, 2064, 384), (130, 60, 272, 128),                                                            # of 128
    (30, 200, 2064, 384), (2, 4100, 2064, 256)])                                                          # of 256
def test_tiles_of_every_size(groups, per, n, k):
    wc, ws, wv = drawn(groups, n, k, seed=per)
    nd = (to_dev(wc), to_dev(ws))
    pk = rp.pack_weights(*nd, fp4=True)
    for i, (dtype, out_dtype, packed) in enumerate(KINDS):
        rng = np.random.default_rng(i)
        off = scattered(groups * per, groups, rng, outside=i % 2)
        say(f"mxfp4_matmul tiles groups={groups} per={per} n={n} k={k} x={dtype} out={out_dtype} packed={packed}")
        x = rng.standard_normal((groups * per, k)) * np.exp(rng.uniform(-2, 2, (groups * per, 1)))
        if dtype is not None:
            t = torch.from_numpy(x.astype(np.float32)).to(dtype)
            x = t.double().numpy()
        xc, xs, xv = fp4(x)
        out = torch.full((groups * per, n), 7.0, dtype=out_dtype, device=DEV)
        w, s = pk if packed else nd
        got = rp.mxfp4_matmul(to_dev(xc) if dtype is None else t.to(DEV), w, s, group_offsets=torch.tensor(
            off, dtype=torch.int32, device=DEV), out=out, x_scales=to_dev(xs) if dtype is None else None,
            weight_format=rp.WEIGHTS_PACKED if packed else rp.WEIGHTS_ND)
        torch.cuda.synchronize()
        check(got, xv, wv, off, out_dtype)
        assert bool((got[:off[0]] == 7).all()) and bool((got[off[-1]:] == 7).all())


@pytest.mark.parametrize("rows", [1, 3, 4, 5])
@pytest.mark.parametrize("values", [False, True])
def test_few_scales_of_a_wide_product(rows, values):
    """One K step and so many channels that the size alone asks for tiles: x has 4 to 20 bytes of
    scales in all, in a tensor of just that size behind others."""
    n, k = 340_016, 128
    wc, ws, wv = drawn(1, n, k, seed=rows)
    rng = np.random.default_rng(rows)
    x = rng.standard_normal((rows, k))
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    xc, xs, xv = fp4(t.double().numpy())
    for packed in (False, True):
        say(f"mxfp4_matmul wide rows={rows} n={n} k={k} values={values} packed={packed}")
        w, s = rp.pack_weights(to_dev(wc), to_dev(ws), fp4=True) if packed else (to_dev(wc), to_dev(ws))
        got = rp.mxfp4_matmul(t.to(DEV) if values else to_dev(xc), w, s, x_scales=None if values else to_dev(xs),
                              out_dtype=torch.float32, weight_format=rp.WEIGHTS_PACKED if packed else rp.WEIGHTS_ND)
        torch.cuda.synchronize()
        check(got, xv, wv, [0, rows], torch.float32)


def uses_tiles(rows, groups, n, k, packed=False):
    """The many-rows kernel is what keeps x's codes in a workspace. (Codes take it from half the size on.)"""
    b = ctypes.c_size_t()
    assert rp.load().moe_mxfp4_matmul_workspace_size(rows, groups, n, k, 2, int(packed), ctypes.byref(b)) == 0
    return b.value > 0


def test_rows_outside_the_groups_are_not_quantised():
    """Rows before the first group and behind the last take no part: x holds NaN there and the
    workspace keeps, but for the codes and scales of the rows inside, what was in it."""
    rows, groups, n, k = 5000, 6, 2048, 512
    lo, hi = 700, 1500
    assert uses_tiles(rows, groups, n, k)
    wc, ws, wv = drawn(groups, n, k, seed=3)
    off = [lo, 800, 800, 1100, 1101, 1300, hi]
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        say(f"mxfp4_matmul rows outside {dtype}")
        x = torch.randn((rows, k), generator=torch.Generator().manual_seed(1)).to(dtype)
        xv = fp4(x[lo:hi].double().numpy())[2]
        x[:lo] = float("nan")
        x[hi:] = float("nan")
        area = torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device=DEV)
        out = torch.full((rows, n), 7.0, device=DEV)
        rp.mxfp4_matmul(x.to(DEV), to_dev(wc), to_dev(ws), group_offsets=torch.tensor(off, dtype=torch.int32, device=DEV),
                        out=out, workspace=area)
        check(out[lo:hi], xv, wv, [o - lo for o in off], torch.float32)
        assert bool((out[:lo] == 7).all()) and bool((out[hi:] == 7).all())
        assert int((area != 0xA5).sum()) <= (hi - lo) * (k // 2 + k // 32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_tiles_quantisation_of_every_16_bit_value(dtype):
    """x against identity weights on the many-rows kernel, as test_quantisation_of_every_bf16_value:
    every finite value of a 16-bit type, also given as fp32, in random groups and in groups of
    neighbouring magnitudes; and against the codes of mx_quantize, bit for bit."""
    k, n = 256, 8192
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    value = torch.from_numpy(bits.astype(np.int16)).view(dtype)
    bits = bits[torch.isfinite(value.float()).numpy()]
    w = np.zeros((1, n, k), dtype=np.uint8)
    w[0, np.arange(n), np.arange(n) % k] = 2
    wc, ws = to_dev(mxfp.pack_fp4(w)), torch.full((1, n, k // 32), 127, dtype=torch.uint8, device=DEV)
    for order in ("random", "sorted"):
        b = np.random.default_rng(1).permutation(bits)
        if order == "sorted":
            b = bits[np.argsort(bits & 0x7fff, kind="stable")]
        b = np.concatenate([b, np.zeros((-b.size) % k, np.uint16)]).reshape(-1, k)
        x = torch.from_numpy(b.astype(np.int16)).view(dtype)
        x = torch.cat([x, x])   # rows enough for tiles
        assert uses_tiles(x.shape[0], 1, n, k)
        c, s = mxfp.quantize(x.double().numpy(), "e2m1")
        want = mxfp.dequantize(c, s, "e2m1")
        normal = np.abs(want) >= 2.0 ** -126
        for given in (dtype, torch.float32):
            say(f"mxfp4_matmul tiles, every {dtype} value as {given}, {order}")
            xd = x.to(given).to(DEV)
            got = rp.mxfp4_matmul(xd, wc, ws, out_dtype=torch.float32)
            codes, scales = rp.mx_quantize(xd, rp.QUANT_MXFP4)
            same = rp.mxfp4_matmul(codes, wc, ws, x_scales=scales, out_dtype=torch.float32)
            assert torch.equal(got, same)
            for part in (got[:, :k], got[:, -k:]):
                part = part.cpu().double().numpy()
                assert np.array_equal(part[normal], want[normal])
                assert np.all(np.abs(part[~normal]) <= 2.0 ** -126)


@pytest.mark.parametrize("rows,groups,n,k", [(520, 1, 8192, 640), (900, 40, 2064, 512), (2100, 3, 2064, 1408)])
def test_tiles_same_result_as_codes(rows, groups, n, k):
    """x quantised in the call gives the bits of the product of mx_quantize's codes (tiles of more
    than one size), with the workspace of the call or a given one, whatever that holds."""
    assert uses_tiles(rows, groups, n, k) and uses_tiles(rows, groups, n, k, packed=True)
    wc, ws, _ = drawn(groups, n, k, seed=rows)
    w, s = to_dev(wc), to_dev(ws)
    off = [0, rows] if groups == 1 else scattered(rows, groups, np.random.default_rng(0), 0)
    off = torch.tensor(off, dtype=torch.int32, device=DEV)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        say(f"mxfp4_matmul tiles against codes rows={rows} groups={groups} {dtype}")
        x = torch.randn((rows, k), generator=torch.Generator().manual_seed(rows)).to(dtype).to(DEV)
        codes, scales = rp.mx_quantize(x, rp.QUANT_MXFP4)
        want = rp.mxfp4_matmul(codes, w, s, x_scales=scales, group_offsets=off, out_dtype=torch.float32)
        assert bool((want != 0).any(dim=1).all())
        area = torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device=DEV)
        for kw in (dict(), dict(workspace=area), dict(workspace=area)):
            assert torch.equal(want, rp.mxfp4_matmul(x, w, s, group_offsets=off, out_dtype=torch.float32, **kw))


def test_tiles_captured_and_replayed_on_two_streams():
    """Two captured graphs whose calls quantise into workspaces of their own, replayed in turn on
    changed inputs with eager calls between, and calls on another stream at the same time."""
    n, k = 2064, 640
    held = []
    for rows, dtype, packed in [(700, torch.float32, False), (1500, torch.bfloat16, True)]:
        assert uses_tiles(rows, 3, n, k, packed)
        wc, ws, _ = drawn(3, n, k, seed=rows)
        w, s = to_dev(wc), to_dev(ws)
        if packed:
            w, s = rp.pack_weights(w, s, fp4=True)
        kw = dict(group_offsets=torch.tensor([0, rows // 4, rows // 4, rows], dtype=torch.int32, device=DEV),
                  weight_format=rp.WEIGHTS_PACKED if packed else rp.WEIGHTS_ND)
        x = torch.randn((rows, k), device=DEV).to(dtype)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            first = [rp.mxfp4_matmul(x, w, s, **kw) for _ in range(3)]
        second = [rp.mxfp4_matmul(x, w, s, **kw) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        for a in first + second:
            assert torch.equal(a, first[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rp.mxfp4_matmul(x, w, s, **kw)
        held.append((graph, x, w, s, kw, out))
    for _ in range(4):
        for graph, x, *_ in held:
            x.copy_(torch.randn_like(x))
            graph.replay()
        eager = [rp.mxfp4_matmul(x, w, s, **kw) for _, x, w, s, kw, _ in held]
        torch.cuda.synchronize()
        for (*_, out), want in zip(held, eager):
            assert torch.equal(out, want)


@pytest.mark.parametrize("rows,groups,n,k", [
    (2048, 8, 4096, 384), (2000, 8, 4096, 128),   # tiles of 128 rows, groups of more: weights read more than once
    (4096, 1, 3600, 256),                         # one dense group, the last channel block partly filled
    (70, 1, 16384, 1024), (190, 3, 16400, 512)])    # dense and grouped, tiles of 64
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_tiles_with_weights_read_more_than_once(rows, groups, n, k, kind):
    dtype, out_dtype, packed = KINDS[kind]
    assert uses_tiles(rows, groups, n, k, packed)
    off = None if groups == 1 else scattered(rows, groups, np.random.default_rng(kind), 0)
    product(rows, groups, n, k, off, dtype, out_dtype, packed, seed=kind)
