"""The norm and its gradient on the GPU against float64.

Bounds (u = 2^-24, the largest relative error of an fp32 rounding; e = finfo(T).eps / 2, that of
one to T, 0 for fp32, whose last product's rounding is counted already; t = half the smallest
subnormal of T):
  h      the fp32 sum rounded to T, exactly;
  rstd   squares summed in 64 bits: one rounding to fp32;
  y      rstd's rounding and two products: 3 u, then T: 3.1 u |y| + e |y| + t, and where h rstd is
         below fp32's smallest normal an absolute 2^-150 |w|;
  codes  those of y's bits by the oracle's quantiser, exactly;
  grad_x with rstd given: xh and a are one product each (u); a thread sums up to 16 terms of a xh,
         64 lanes and 16 waves are joined: 16 + 6 + 16 additions and the division, so sum(a xh) / C
         is off by at most D = 42 u sum|a xh| / C; rstd (a - xh dot) + grad_h then takes up to 5
         more roundings of each term: 5 u rstd (|a| + |xh dot|) + rstd |xh| D + u |grad_x|, then T;
  grad_w a thread adds at most rows / 256 + 1 rows (narrow ones: rows / 4096 + 1), 16 of them, up to
         32 parts and 5 pairs of sums are joined: rows / 256 + 54 additions, no more than the
         rows / 512 + 68 allowed, u sum|grad_y xh| each, up to 7168 rows."""
import numpy as np
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say
from oracle import dense, mxfp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
TYPES = [torch.bfloat16, torch.float16, torch.float32]
FORMATS = [(rp.QUANT_E4M3, "e4m3"), (rp.QUANT_E5M2, "e5m2"), (rp.QUANT_MXFP4, "e2m1")]


def to_t(dtype):
    """(e, t): the relative and the absolute half step of a rounding to dtype."""
    f = torch.finfo(dtype)
    return (0.0 if dtype == torch.float32 else f.eps / 2), f.smallest_normal * f.eps / 2


def rows_of(rows, cols, dtype, seed=0, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    scale = torch.exp(torch.rand((rows, 1), generator=gen) * 2 * spread - spread)
    return (torch.randn((rows, cols), generator=gen) * scale).to(dtype)


def weight_of(cols, dtype, seed=1):
    return (1.0 + 0.3 * torch.randn((cols,), generator=torch.Generator().manual_seed(seed))).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check_norm(x, residual, w, got, eps=EPS):
    y, h, rstd, codes, scales = got
    dtype = x.dtype
    want_h = x if residual is None else (x.float() + residual.float()).to(dtype)
    assert torch.equal(h.cpu(), want_h)
    want, r = dense.rms_norm(f64(want_h), f64(w), eps)
    assert np.all(np.abs(f64(rstd) / r - 1) <= U * 1.001)
    e, t = to_t(dtype)
    err = 3.1 * U * np.abs(want) + 2.0 ** -150 * np.maximum(np.abs(f64(w)), 1.0)
    bound = err + e * (np.abs(want) + err) + t
    assert np.all(np.abs(f64(y) - want) <= bound)


def on(t, off=0):
    """t on the GPU, `off` elements behind a 16-byte boundary."""
    if t is None:
        return None
    buf = torch.empty((t.numel() + 8,), dtype=t.dtype, device=DEV)
    out = buf[off:off + t.numel()].view(t.shape)
    out.copy_(t)
    return out


# columns at the edges of each number of lanes a row, and odd ones
COLS = [1, 7, 8, 31, 100, 128, 129, 500, 512, 520, 1001, 1024, 2047, 2048, 4096, 4104, 7168, 8192, 8200, 16383, 16384]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(cols, dtype):
    for rows, residual, wt, off in [(1, True, dtype, 0), (17, False, torch.float32, 0), (34, True, torch.float32, 0),
                                    (5, True, dtype, 3)]:
        say(f"rms_norm {rows}x{cols} {dtype} residual={residual} weight={wt} offset={off}")
        x, w = rows_of(rows, cols, dtype), weight_of(cols, wt)
        r = rows_of(rows, cols, dtype, seed=2) if residual else None
        got = rp.rms_norm(on(x, off), on(w), on(r, off), eps=EPS)
        assert got[3] is None and got[4] is None
        check_norm(x, r, w, got)


@pytest.mark.parametrize("cols", [32, 96, 128, 160, 512, 1056, 2048, 7168, 8224, 16384])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode,fmt", FORMATS)
def test_codes(cols, dtype, mode, fmt):
    for rows, off in [(1, 0), (19, 0), (6, 5)]:
        say(f"rms_norm {rows}x{cols} {dtype} {fmt} offset={off}")
        x, r, w = rows_of(rows, cols, dtype), rows_of(rows, cols, dtype, seed=2), weight_of(cols, dtype)
        x[0, :32] = 0
        r[0, :32] = 0   # a group of zeros
        got = rp.rms_norm(on(x, off), on(w), on(r, off), eps=EPS, quant_mode=mode)
        check_norm(x, r, w, got)
        c, s = mxfp.quantize(f64(got[0]), fmt)
        c = mxfp.pack_fp4(c) if fmt == "e2m1" else c
        assert np.array_equal(got[3].cpu().numpy(), c)
        assert np.array_equal(got[4].cpu().numpy()[:, :cols // 32], s[:, :cols // 32])
        assert got[4].shape[1] == rp.mx_scale_cols(cols) and not got[4][:, cols // 32:].any()
        q, qs = rp.mx_quantize(got[0], mode)
        assert torch.equal(q, got[3]) and torch.equal(qs, got[4])
        alone = rp.rms_norm(on(x, off), on(w), on(r, off), eps=EPS, quant_mode=mode, want_y=False)
        assert alone[0] is None and all(torch.equal(a, b) for a, b in zip(alone[1:], got[1:]))


def test_extremes():
    """Rows of zeros; of the largest finite values, whose squares no fp32 holds; of subnormals;
    and rows with infinities and NaN, which the formula makes NaN and which touch no other row."""
    for dtype, big in [(torch.float32, 3e38), (torch.bfloat16, 3e38), (torch.float16, 65504.0)]:
        tiny = float(torch.finfo(dtype).smallest_normal) / 4
        # (linspace's step overflows to infinity at 3e38: that row is NaN from its second element on)
        x = torch.stack([torch.zeros(256), torch.full((256,), big), torch.full((256,), tiny), torch.linspace(-big, big, 256),
                         torch.ones(256), torch.linspace(-1, 1, 256) * big]).to(dtype)
        w = weight_of(256, dtype)
        got = rp.rms_norm(on(x), on(w), eps=EPS)
        y, r = dense.rms_norm(f64(x), f64(w), EPS)
        # rstd of the largest rows is a subnormal fp32: half its step, 2^-150, on top
        within = lambda a, b, bound: np.all((np.abs(a - b) <= bound) | (np.isnan(a) & np.isnan(b)))  # noqa: E731
        assert within(f64(got[2]), r, U * 1.001 * r + 2.0 ** -150)
        e, t = to_t(dtype)
        err = np.abs(y) * (3.1 * U + 2.0 ** -150 / r[:, None]) + 2.0 ** -150 * 3
        assert within(f64(got[0]), y, err + e * (np.abs(y) + err) + t)
        bad = x.clone()
        bad[0, 3], bad[2, 200], bad[3, 0] = float("inf"), float("nan"), -float("inf")
        again = rp.rms_norm(on(bad), on(w), eps=EPS)
        for row in (1, 4, 5):
            assert torch.equal(again[0][row], got[0][row]) and again[2][row] == got[2][row]
        assert bool(again[0][2].isnan().all()) and bool(again[0][0, 3].isnan()) and bool(again[0][3, 0].isnan())
        assert float(again[2][0]) == 0 and bool((again[0][0, 4:] == 0).all())


def check_backward(gy, h, w, rstd, gh, got):
    gx, gw = got
    want, want_w = dense.rms_norm_backward(f64(gy), f64(h), f64(w), f64(rstd), None if gh is None else f64(gh))
    r = f64(rstd)[:, None]
    xh, a = f64(h) * r, f64(gy) * f64(w)
    C = h.shape[1]
    dot, mag = (a * xh).sum(1, keepdims=True) / C, np.abs(a * xh).sum(1, keepdims=True) / C
    e, t = to_t(h.dtype)
    err = 5 * U * r * (np.abs(a) + np.abs(xh * dot)) + r * np.abs(xh) * 42 * U * mag + U * np.abs(want) + 2.0 ** -140
    assert np.all(np.abs(f64(gx) - want) <= err + e * (np.abs(want) + err) + t)
    bound = (h.shape[0] / 512 + 68) * U * np.abs(f64(gy) * xh).sum(0) + 2.0 ** -140
    assert gw.dtype == torch.float32 and np.all(np.abs(f64(gw) - want_w) <= bound)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(cols, dtype):
    for rows, with_h, wt, off in [(1, True, dtype, 0), (17, False, torch.float32, 0), (1100, True, dtype, 0),
                                  (5, True, torch.float32, 3)]:
        say(f"rms_norm_backward {rows}x{cols} {dtype} grad_h={with_h} weight={wt} offset={off}")
        h, w = rows_of(rows, cols, dtype), weight_of(cols, wt)
        gy, gh = rows_of(rows, cols, dtype, seed=3), rows_of(rows, cols, dtype, seed=4) if with_h else None
        rstd = torch.from_numpy(dense.rms_norm(f64(h), f64(w), EPS)[1]).float()
        got = rp.rms_norm_backward(on(gy, off), on(h, off), on(w), on(rstd), grad_h=on(gh, off))
        check_backward(gy, h, w, rstd, gh, got)
        again = rp.rms_norm_backward(on(gy, off), on(h, off), on(w), on(rstd), grad_h=on(gh, off))
        assert all(torch.equal(a, b) for a, b in zip(got, again))   # a fixed order


def test_backward_against_differences():
    """The gradients of sum(y g) + sum(h q) by central differences of the norm itself, in fp32 along
    random directions: the loss's rounding (2^-20 of its terms over the step) and the third
    derivative are far below 1e-2 of the directions' gradients, which are of the order 1."""
    rows, cols, d = 3, 96, 2.0 ** -6
    x, r, w = rows_of(rows, cols, torch.float32, spread=0.1), rows_of(rows, cols, torch.float32, 2, 0.1), weight_of(cols, torch.float32)
    g, q = rows_of(rows, cols, torch.float32, 3, 0.1), rows_of(rows, cols, torch.float32, 4, 0.1)

    def loss(x, r, w):
        y, h, _, _, _ = rp.rms_norm(on(x), on(w), on(r), eps=EPS)
        return float((f64(y) * f64(g)).sum() + (f64(h) * f64(q)).sum())

    _, h, rstd, _, _ = rp.rms_norm(on(x), on(w), on(r), eps=EPS)
    gx, gw = rp.rms_norm_backward(on(g), h, on(w), rstd, grad_h=on(q))
    for seed in range(4):
        vx, vw = rows_of(rows, cols, torch.float32, 10 + seed, 0.1), weight_of(cols, torch.float32, 20 + seed) - 1
        for along, got in (((vx * d, None, None), (f64(gx) * f64(vx)).sum()), ((None, vx * d, None), (f64(gx) * f64(vx)).sum()),
                           ((None, None, vw * d), (f64(gw) * f64(vw)).sum())):
            up = [t if v is None else t + v for t, v in zip((x, r, w), along)]
            down = [t if v is None else t - v for t, v in zip((x, r, w), along)]
            assert abs((loss(*up) - loss(*down)) / (2 * d) - got) <= 1e-2 * max(1.0, abs(got))


def test_no_rows():
    x, w = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV), torch.ones(64, dtype=torch.bfloat16, device=DEV)
    y, h, rstd, codes, scales = rp.rms_norm(x, w, x, quant_mode=rp.QUANT_E4M3)
    assert y.shape == h.shape == (0, 64) and rstd.shape == (0,) and codes.shape == (0, 64) and scales.shape == (0, 2)
    gx, gw = rp.rms_norm_backward(x, x, w, rstd)
    assert gx.shape == (0, 64) and not gw.any()


def test_many_rows():
    """More rows than one launch has blocks for: rows of one repeating pattern, so each row's result is known."""
    rows, cols = (1 << 24) - 2, 8
    base = rows_of(16, cols, torch.bfloat16)
    w = weight_of(cols, torch.bfloat16)
    want = rp.rms_norm(on(base), on(w))
    x = on(base).repeat(rows // 16 + 1, 1)[:rows].contiguous()
    y, _, rstd, _, _ = rp.rms_norm(x, on(w))
    full = rows // 16 * 16
    assert bool((y[:full].view(-1, 16, cols) == want[0]).all()) and bool((rstd[:full].view(-1, 16) == want[2]).all())
    assert torch.equal(y[full:], want[0][:rows - full])
    gx, gw = rp.rms_norm_backward(y, x, on(w), rstd)
    one = rp.rms_norm_backward(want[0], on(base), on(w), want[2])
    assert bool((gx[:full].view(-1, 16, cols) == one[0]).all())
    # the weight's gradient: full / 16 times that of the pattern, and the last rows'
    xh = f64(base) * f64(want[2])[:, None]
    terms = f64(want[0]) * xh
    want_w = terms.sum(0) * (rows // 16) + terms[:rows - full].sum(0)
    mag = np.abs(terms).sum(0) * (rows // 16 + 1)
    assert np.all(np.abs(f64(gw) - want_w) <= (rows / 512 + 68) * U * mag)


def test_captured_replayed_and_two_streams():
    x, r, w = (on(rows_of(300, 2048, torch.bfloat16, s)) for s in range(3))
    w = w[0].contiguous()
    g = on(rows_of(300, 2048, torch.bfloat16, 5))

    def step(x, r, g):
        y, h, rstd, codes, scales = rp.rms_norm(x, w, r, quant_mode=rp.QUANT_E4M3)
        return y, h, rstd, codes, scales, *rp.rms_norm_backward(g, h, w, rstd, grad_h=y)

    step(x, r, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, r, g)
    for seed in range(3):
        for t, k in ((x, 0), (r, 1), (g, 2)):
            t.copy_(rows_of(300, 2048, torch.bfloat16, 10 * seed + k))
        graph.replay()
        want = step(x.clone(), r.clone(), g.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([step(x, r, g) for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for runs in got for run in runs for a, b in zip(run, want))


def test_in_place_gradients():
    """The C call with grad_x in the place of grad_y and of grad_h, as its documentation allows."""
    lib = rp.load()
    for dtype, code in [(torch.bfloat16, 2), (torch.float32, 0)]:
        h, gy, gh = (on(rows_of(40, 1000, dtype, s)) for s in (0, 3, 4))
        w = on(weight_of(1000, dtype))
        _, _, rstd, _, _ = rp.rms_norm(h, w)
        want = rp.rms_norm_backward(gy, h, w, rstd, grad_h=gh)
        ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
        for place in range(2):
            a, b = gy.clone(), gh.clone()
            gw = torch.empty(1000, device=DEV)
            assert lib.moe_rms_norm_backward(a.data_ptr(), h.data_ptr(), b.data_ptr(), code, 40, 1000, w.data_ptr(), code,
                                             rstd.data_ptr(), (a, b)[place].data_ptr(), gw.data_ptr(), ws.data_ptr(),
                                             ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
            torch.cuda.synchronize()
            assert torch.equal((a, b)[place], want[0]) and torch.equal(gw, want[1])


@pytest.mark.parametrize("cols", [100, 500, 1001, 2048, 7168, 8200, 16384])
@pytest.mark.parametrize("dtype", TYPES)
def test_blocks_of_many_rows(cols, dtype):
    """More rows than there are blocks, so that a block loads one while it sums another; codes of them, too."""
    x, r, w = rows_of(2600, cols, dtype), rows_of(2600, cols, dtype, 2), weight_of(cols, dtype)
    say(f"rms_norm 2600x{cols} {dtype}")
    check_norm(x, r, w, rp.rms_norm(on(x), on(w), on(r)))
    y, h, rstd, codes, scales = rp.rms_norm(on(x), on(w), on(r), quant_mode=rp.QUANT_E4M3) if cols % 32 == 0 else (None,) * 5
    if codes is not None:
        check_norm(x, r, w, (y, h, rstd, codes, scales))
        want_codes, want_scales = rp.mx_quantize(y, quant_mode=rp.QUANT_E4M3)
        assert torch.equal(codes, want_codes.view(torch.uint8)) and torch.equal(scales, want_scales.view(torch.uint8))


@pytest.mark.parametrize("rows,cols,dtype", [(16500, 7168, torch.bfloat16), (30000, 2048, torch.float32),
                                             (270000, 8200, torch.bfloat16)])
def test_large(rows, cols, dtype):
    """Outputs larger than the cache, and of more than 2^31 elements: every row as in a small call."""
    say(f"rms_norm {rows}x{cols} {dtype}")
    gen = torch.Generator(device=DEV).manual_seed(0)
    x, r = (torch.empty((rows, cols), dtype=dtype, device=DEV).normal_(0, 1, generator=gen) for _ in range(2))
    w = on(weight_of(cols, dtype))
    y, h, rstd, _, _ = rp.rms_norm(x, w, r)
    gx, gw = rp.rms_norm_backward(x, h, w, rstd, grad_h=r)
    want_w, mag = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    for lo in range(0, rows, 5000):
        some = slice(lo, lo + 5000)
        part = rp.rms_norm(x[some], w, r[some])
        assert torch.equal(y[some], part[0]) and torch.equal(h[some], part[1]) and torch.equal(rstd[some], part[2]), lo
        assert torch.equal(gx[some], rp.rms_norm_backward(x[some], h[some], w, rstd[some], grad_h=r[some])[0]), lo
        terms = x[some].double() * (h[some].double() * rstd[some].double()[:, None])
        want_w += terms.sum(0)
        mag += terms.abs().sum(0)
    assert bool(((gw.double() - want_w).abs() <= (rows / 256 + 54) * U * mag).all())


@pytest.mark.parametrize("rows,cols", [(2600, 1000), (2600, 100), (700, 7168), (700, 8200), (40, 1001)])
def test_in_place(rows, cols):
    """The C calls with an output in an input's place, as the documentation allows, with more rows than blocks."""
    lib, stream = rp.load(), torch.cuda.current_stream().cuda_stream
    for dtype, code in [(torch.bfloat16, 2), (torch.float32, 0)]:
        x, r = on(rows_of(rows, cols, dtype)), on(rows_of(rows, cols, dtype, 2))
        w = on(weight_of(cols, dtype))
        y, h, rstd, _, _ = rp.rms_norm(x, w, r)
        for y_at in range(2):
            a, b, got = x.clone(), r.clone(), torch.empty_like(rstd)
            yp, hp = ((a, b), (b, a))[y_at]
            assert lib.moe_rms_norm(a.data_ptr(), b.data_ptr(), code, rows, cols, w.data_ptr(), code, EPS, -1, yp.data_ptr(),
                                    hp.data_ptr(), got.data_ptr(), None, None, stream) == 0
            assert torch.equal(yp, y) and torch.equal(hp, h) and torch.equal(got, rstd)
        want = rp.rms_norm_backward(y, h, w, rstd, grad_h=r)
        ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
        a, gw = h.clone(), torch.empty(cols, device=DEV)
        assert lib.moe_rms_norm_backward(y.data_ptr(), a.data_ptr(), r.data_ptr(), code, rows, cols, w.data_ptr(), code,
                                         rstd.data_ptr(), a.data_ptr(), gw.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
        assert torch.equal(a, want[0]) and torch.equal(gw, want[1])
