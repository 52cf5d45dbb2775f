"""The 16-bit products by every tile of the LDS-staged kernel, in every form: whole and odd rows, both element
types and both output types, outputs at a 16-byte boundary and not, with and without items that blocks share,
a block with one item and with several. All of an output is compared with float64 on the GPU (the bound of
test_gpu_gmm16), what lies around it and the rows outside the groups have to stay as they were, and the
workspace of shared items has to be used where the case says that items are shared."""
import functools

import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gmm16_cases import MANY_ITEMS, cases, offsets
from gpu_support import DEV, say

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
GUARD = 4096   # elements in front of and behind an output


def normal(shape, dtype, gen, std):
    """Normal values whose rows differ in size by up to e^4."""
    t = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    t.mul_(torch.exp(torch.rand((*shape[:-1], 1), generator=gen, device=DEV) * 4 - 2) * std)
    return t.to(dtype)


def guarded(shape, dtype, off):
    """A tensor of 7s, `off` elements behind a 16-byte boundary, and the buffer around it."""
    size = functools.reduce(lambda a, b: a * b, shape)
    buf = torch.full((size + 2 * GUARD,), 7.0, dtype=dtype, device=DEV)
    return buf[GUARD + off:GUARD + off + size].view(shape), buf


def around_is_kept(buf, size, off):
    return bool((buf[:GUARD + off] == 7).all()) and bool((buf[GUARD + off + size:] == 7).all())


def close(got, want, mag, length, dtype):
    """The largest error over the bound of test_gpu_gmm16."""
    err = mag * ((length / 16 + 64) * 2.0 ** -23)
    f = torch.finfo(dtype)
    e, t = (0.0, 0.0) if dtype == FP else (f.eps / 2, f.smallest_normal * f.eps / 2)
    bound = err + e * (want.abs() + err) + t + 2.0 ** -120
    return float(((got.double() - want).abs() / bound).max()) if got.numel() else 0.0   # (NaN is not <= 1)


def references(form, a, b, spans):
    """(want, sum of magnitudes) of each group in float64."""
    for g, (lo, hi) in enumerate(spans):
        if form == "weights":
            x, y = a[lo:hi].double().t().contiguous(), b[lo:hi].double()
        else:
            x, y = a[lo:hi].double(), b[g].double()
            if form == "forward":
                y = y.t().contiguous()
        yield g, lo, hi, x @ y, x.abs() @ y.abs()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form,tile,shared,rows,groups,n,k", cases())
def test_tile(form, tile, shared, rows, groups, n, k, dtype):
    say(f"{form} tile {tile} shared={shared}: {rows} rows, {groups} groups, n {n}, k {k}, {dtype}")
    gen = torch.Generator(device=DEV).manual_seed(rows + n + k)
    ends = offsets(rows, groups)
    spans = [(0, rows)] if ends is None else list(zip(ends[:-1], ends[1:]))
    o = None if ends is None else torch.tensor(ends, dtype=torch.int32, device=DEV)
    if form == "weights":
        a, b = normal((rows, n), dtype, gen, 1.0), normal((rows, k), dtype, gen, 1.0)
        shape, need = (groups, n, k), rp._sized("moe_grouped_matmul_wgrad_workspace_size", rows, groups, n, k)
    else:
        trans = form == "transposed"
        a = normal((rows, k), dtype, gen, 1.0)
        b = normal((groups, k, n) if trans else (groups, n, k), dtype, gen, k ** -0.5)
        shape, need = (rows, n), rp._sized("moe_grouped_matmul_workspace_size", rows, groups, n, k, int(trans))
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)

    def call(out_dtype, off):
        out, buf = guarded(shape, out_dtype, off)
        ws.fill_(255)
        if form == "weights":
            rp.grouped_matmul_wgrad(a, b, o, out=out if ends is not None else out[0], workspace=ws)
        else:
            rp.grouped_matmul(a, b, o, transpose_w=trans, out=out, workspace=ws)
        assert around_is_kept(buf, out.numel(), off), (out_dtype, off)
        if shared:   # (the parts lie first in the workspace; 255s are NaN)
            assert bool((ws[:256 * tile * (256 if tile > 64 else 128) * 4] != 255).any())
        return out

    calls = [(dtype, 0), (FP, 0), (dtype, 1), (FP, 3)]
    outs = [call(*c) for c in calls]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])   # wherever they lie
    for g, lo, hi, want, mag in references(form, a, b, spans):
        for (out_dtype, _), out in zip(calls[:2], outs):
            got = out[g] if form == "weights" else out[lo:hi]
            worst = close(got, want, mag, hi - lo if form == "weights" else k, out_dtype)
            assert worst <= 1.0, (g, out_dtype, worst)
    if form != "weights":   # rows outside the groups
        for out in outs:
            assert bool((out[:spans[0][0]] == 7).all()) and bool((out[spans[-1][1]:] == 7).all())


@pytest.mark.parametrize("form,tile,each,groups,n,k", MANY_ITEMS)
def test_many_items(form, tile, each, groups, n, k):
    """Blocks with more items than they describe at a time: whole numbers, whose sums fp32 holds exactly."""
    say(f"{form} tile {tile}: {groups} groups of {each} rows, n {n}, k {k}")
    gen = torch.Generator(device=DEV).manual_seed(0)
    draw = lambda *s: torch.randint(-7, 8, s, generator=gen, device=DEV).to(BF)  # noqa: E731
    o = torch.arange(0, each * groups + 1, each, dtype=torch.int32, device=DEV)
    if form == "weights":
        a, b = draw(groups * each, n), draw(groups * each, k)
        got = rp.grouped_matmul_wgrad(a, b, o)
        want = torch.bmm(a.float().view(groups, each, n).transpose(1, 2).contiguous(), b.float().view(groups, each, k))
        assert torch.equal(got, want.to(BF))
        return
    trans = form == "transposed"
    x, w = draw(groups * each, k), draw(groups, k, n) if trans else draw(groups, n, k)
    got = rp.grouped_matmul(x, w, o, transpose_w=trans)
    right = w.float() if trans else w.float().transpose(1, 2).contiguous()
    assert torch.equal(got.view(groups, each, n), torch.bmm(x.float().view(groups, each, k), right).to(BF))
