"""Outputs inside larger buffers, at every element of a 16-byte piece: nothing in front of them or behind
them is written, and their values are as good as those of an output of its own. The products by the kernels of
few rows and of any address (test_gpu_gmm16_tiles has the others), the norm and its gradient through the C
calls, within the bounds of test_gpu_gmm16 and test_gpu_norm."""
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say
from oracle import dense
from test_gpu_gmm16 import BF, FP, HF, check, f64, on, values
from test_gpu_gmm16_tiles import around_is_kept, guarded
from test_gpu_norm import check_backward, check_norm

pytestmark = pytest.mark.gpu


def moved(t, off):
    """t, `off` elements behind a 16-byte boundary."""
    return on(t.cpu(), off)


@pytest.mark.parametrize("out_dtype", [BF, FP])
@pytest.mark.parametrize("rows,groups,n,k", [(1, 1, 8, 64), (7, 1, 61, 72), (16, 3, 64, 100), (30, 1, 9, 512), (70, 1, 8, 64)])
def test_few_rows(rows, groups, n, k, out_dtype):
    """The kernel of few rows, forward; and the same operands at an odd element."""
    say(f"few rows {rows} {groups} {n} {k} {out_dtype}")
    x, w = on(values((rows, k), BF, 0)), on(values((groups, n, k), BF, 1))
    o = None if groups == 1 else torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device=DEV)
    want = rp.grouped_matmul(x, w, o, out_dtype=out_dtype)
    for off in range(8):
        out, buf = guarded((rows, n), out_dtype, off)
        rp.grouped_matmul(x, w, o, out=out)
        assert torch.equal(out, want) and around_is_kept(buf, out.numel(), off)
        out, buf = guarded((rows, n), out_dtype, off)
        rp.grouped_matmul(moved(x, 1), moved(w, 3), o, out=out)
        assert torch.equal(out, want) and around_is_kept(buf, out.numel(), off)


@pytest.mark.parametrize("form", ["forward", "transposed", "weights"])
@pytest.mark.parametrize("n,k", [(64, 128), (61, 131), (8, 264)])
def test_operands_at_any_element(form, n, k):
    """Operands at an odd element: the kernel for every address, but for odd rows of both, which are copied."""
    rows, o = 130, torch.tensor([0, 50, 50, 129], dtype=torch.int32, device=DEV)
    for out_dtype in (HF, FP):
        say(f"any element {form} {n} {k} {out_dtype}")
        a = moved(values((rows, n if form == "weights" else k), HF, 0), 1)
        b = moved(values((rows, k) if form == "weights" else (3, k, n) if form == "transposed" else (3, n, k), HF, 1), 5)
        results = []
        for off in range(8):
            out, buf = guarded((3, n, k) if form == "weights" else (rows, n), out_dtype, off)
            if form == "weights":
                rp.grouped_matmul_wgrad(a, b, o, out=out)
            else:
                rp.grouped_matmul(a, b, o, transpose_w=form == "transposed", out=out)
            assert around_is_kept(buf, out.numel(), off)
            results.append(out.clone())
        assert all(torch.equal(r, results[0]) for r in results)
        if form == "weights":
            want, mag = dense.grouped_matmul_wgrad(f64(a), f64(b), [0, 50, 50, 129])
            check(results[0], want, mag, 79, out_dtype)
        else:
            want, mag = dense.grouped_matmul(f64(a), f64(b), [0, 50, 50, 129], form == "transposed")
            check(results[0][:129], want[:129], mag[:129], k, out_dtype)
            assert bool((results[0][129:] == 7).all())


def code_of(t):
    return {FP: 0, HF: 1, BF: 2}[t]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (3, 101), (17, 520), (9, 1001), (4, 8224), (2, 16384), (2600, 64)])
def test_norm(rows, cols, dtype):
    """Rows, weight and outputs at 0 to 7 elements from a 16-byte boundary (fp32 rows at 4: 16 bytes but not 32),
    each within its buffer; codes at multiples of 8 bytes, scales at any."""
    say(f"norm bounds {rows}x{cols} {dtype}")
    lib, stream = rp.load(), torch.cuda.current_stream().cuda_stream
    x, r, w = values((rows, cols), dtype, 0), values((rows, cols), dtype, 1), values((cols,), dtype, 2) + 1
    quant = rp.QUANT_E4M3 if cols % 32 == 0 else rp.QUANT_NONE
    for off in range(8):
        y, yb = guarded((rows, cols), dtype, off)
        h, hb = guarded((rows, cols), dtype, off)
        rstd, rb = guarded((rows,), FP, off)
        codes, cb = guarded((rows, cols), torch.uint8, 8 * off)
        scales, sb = guarded((rows, rp.mx_scale_cols(cols)), torch.uint8, off)
        xo, wo, ro = on(x, off), on(w, off), on(r, off)
        assert lib.moe_rms_norm(xo.data_ptr(), ro.data_ptr(), code_of(dtype), rows, cols, wo.data_ptr(), code_of(dtype), 1e-6,
                                quant, y.data_ptr(), h.data_ptr(), rstd.data_ptr(), codes.data_ptr() if quant > 0 else None,
                                scales.data_ptr() if quant > 0 else None, stream) == 0
        torch.cuda.synchronize()
        check_norm(x, r, w, (y, h, rstd, None, None))
        if quant > 0:
            q, qs = rp.mx_quantize(moved(y, 0), quant)
            assert torch.equal(codes, q.view(torch.uint8)) and torch.equal(scales, qs.view(torch.uint8)), off
        for t, b, o in ((y, yb, off), (h, hb, off), (rstd, rb, off), (codes, cb, 8 * off), (scales, sb, off)):
            assert around_is_kept(b, t.numel(), o), off


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 101), (17, 520), (9, 1001), (4, 8224), (2, 16384), (2600, 64)])
def test_norm_backward(rows, cols, dtype):
    say(f"norm gradient bounds {rows}x{cols} {dtype}")
    lib, stream = rp.load(), torch.cuda.current_stream().cuda_stream
    gy, h, gh = (values((rows, cols), dtype, s) for s in range(3))
    w = values((cols,), FP, 3) + 1
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    need = rp._sized("moe_rms_norm_backward_workspace_size", rows, cols)
    for off in range(8):
        gx, xb = guarded((rows, cols), dtype, off)
        gw, wb = guarded((cols,), FP, off)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
        gyo, ho, gho, wo, ro = on(gy, off), on(h, off), on(gh, off), on(w, off), on(rstd, off)
        assert lib.moe_rms_norm_backward(gyo.data_ptr(), ho.data_ptr(), gho.data_ptr(), code_of(dtype), rows, cols,
                                         wo.data_ptr(), 0, ro.data_ptr(), gx.data_ptr(), gw.data_ptr(), ws.data_ptr(), need,
                                         stream) == 0
        torch.cuda.synchronize()
        check_backward(gy, h, w, rstd, gh, (gx, gw))
        for t, b in ((gx, xb), (gw, wb)):
            assert around_is_kept(b, t.numel(), off), off
        assert bool((ws[need:] == 255).all()), off   # nor behind the workspace
