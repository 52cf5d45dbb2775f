"""The 16-bit products of values at the ends of their types, by the kernel of few rows, small and large tiles,
shared items and operands at any address: sums that fp32 holds exactly, so every output is known to the bit."""
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say
from test_gpu_gmm16 import BF, FP, HF, on

pytestmark = pytest.mark.gpu

# (form, rows, n, k, elements from a 16-byte boundary): few rows, tiles of 32 and more rows, shared items, any address
CASES = [("forward", 3, 24, 72, 0), ("forward", 3, 24, 72, 1), ("forward", 100, 136, 200, 0), ("forward", 2100, 1032, 264, 0),
         ("forward", 97, 1032, 1544, 0), ("forward", 40, 72, 264, 3), ("transposed", 3, 24, 72, 0),
         ("transposed", 100, 136, 200, 0), ("transposed", 2100, 1032, 264, 0), ("transposed", 97, 1032, 1544, 0),
         ("transposed", 40, 72, 264, 3), ("weights", 200, 24, 72, 0), ("weights", 512, 3080, 264, 0),
         ("weights", 1537, 40, 72, 0), ("weights", 264, 40, 72, 3)]


def call(form, a, b, out_dtype, off):
    a, b = on(a, off), on(b, off)
    if form == "weights":
        return rp.grouped_matmul_wgrad(a, b, out_dtype=out_dtype)
    return rp.grouped_matmul(a, b, transpose_w=form == "transposed", out_dtype=out_dtype)


def operands(form, rows, n, k, seed, top):
    """Whole numbers from -top to top, and their product in 64 bits: a, b, want."""
    gen = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randint(-top, top + 1, s, generator=gen).double()  # noqa: E731
    if form == "weights":
        a, b = draw(rows, n), draw(rows, k)
        return a, b, a.T @ b
    a, b = draw(rows, k), draw(k, n) if form == "transposed" else draw(n, k)
    return a, b, a @ (b if form == "transposed" else b.T)


@pytest.mark.parametrize("form,rows,n,k,off", CASES)
def test_subnormal_operands(form, rows, n, k, off):
    """Whole multiples of the smallest subnormal of a type times whole numbers: sums of at most 1544 products of 7 x 7
    times a power of two, exact in fp32; nothing counts as zero."""
    a, b, want = operands(form, rows, n, k, 0, 7)
    for dtype, small, large in ((HF, 2.0 ** -24, 1.0), (HF, 1.0, 2.0 ** -24), (BF, 2.0 ** -133, 2.0 ** 60), (BF, 2.0 ** 60, 2.0 ** -133)):
        say(f"subnormals {form} {rows} {n} {k} offset {off} {dtype} {small:g} {large:g}")
        x, y = (a * small).to(dtype), (b * large).to(dtype)
        assert torch.equal(x.double(), a * small) and torch.equal(y.double(), b * large)
        got = call(form, x, y, FP, off)
        assert torch.equal(got.cpu().double(), want * small * large)


@pytest.mark.parametrize("form,rows,n,k,off", CASES)
def test_outputs_of_each_type(form, rows, n, k, off):
    """Sums of whole numbers as fp16 and bf16: rounded to nearest, ties to even, past fp16's largest value to
    infinity; and as fp16's subnormals."""
    a, b, want = operands(form, rows, n, k, 1, 7)
    for dtype, scale in ((HF, 1.0), (BF, 1.0), (HF, 8.0), (HF, 2.0 ** -10)):
        say(f"outputs {form} {rows} {n} {k} offset {off} {dtype} {scale:g}")
        got = call(form, (a * scale).to(dtype), (b * scale).to(dtype), dtype, off)
        exact = (want * scale * scale).to(FP)
        assert torch.equal(exact.double(), want * scale * scale)
        assert torch.equal(got.cpu(), exact.to(dtype))


@pytest.mark.parametrize("form,rows,n,k,off", CASES)
def test_infinities(form, rows, n, k, off):
    """An infinite element meets its own row's or channel's outputs: infinite with the sign of its partner, NaN
    where that is zero; the rest is as without it."""
    a, b, want = operands(form, rows, n, k, 2, 3)
    x, y = a.to(BF), b.to(BF)
    if form == "weights":
        x[5, 1] = float("inf")            # row 5 of b is its partner, output row 1 meets it
        partner, row = y[5], 1
    else:
        x[2, 5] = float("inf")
        partner, row = y[5] if form == "transposed" else y[:, 5], 2
    got = call(form, x, y, FP, off).cpu()
    keep = torch.arange(got.shape[0]) != row
    assert torch.equal(got[keep].double(), want[keep])
    zero = partner == 0
    assert bool(got[row][zero].isnan().all()) and torch.equal(got[row][~zero], torch.sign(partner[~zero].float()) * float("inf"))


def test_one_tensor_as_both_operands():
    """x^T x: both operands of the gradient by w are one tensor."""
    a = torch.randint(-7, 8, (700, 136), generator=torch.Generator().manual_seed(0)).double()
    x = on(a.to(BF))
    assert torch.equal(rp.grouped_matmul_wgrad(x, x, out_dtype=FP).cpu().double(), a.T @ a)
    assert torch.equal(rp.grouped_matmul(x, x, out_dtype=FP).cpu().double(), a @ a.T)


def test_first_calls_inside_a_capture():
    """Calls whose sizes no other test takes, captured without having run before, and replayed on new values."""
    say("first calls inside a capture")
    x, w = torch.zeros((1537, 328), dtype=HF, device=DEV), torch.zeros((6160, 328), dtype=HF, device=DEV)
    g = torch.zeros((1537, 6160), dtype=HF, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, back, gw = rp.grouped_matmul(x, w), rp.grouped_matmul(g, w, transpose_w=True), rp.grouped_matmul_wgrad(g, x)
    for seed in range(3):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        for t in (x, w, g):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = rp.grouped_matmul(x, w), rp.grouped_matmul(g, w, transpose_w=True), rp.grouped_matmul_wgrad(g, x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, back, gw), want))
