"""Host-side refusals of the norm and of the 16-bit products: wrong arguments return an error with a
message before any launch, so these run without a GPU."""
import ctypes
import time
import os

import pytest
import torch

import routing_permute_mxfp8_amd as rp

FAKE = 0x1000   # never dereferenced: every call below fails validation or has nothing to do


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rp.lib_path()):
        from routing_permute_mxfp8_amd import build
        build.build()
    return rp.load()


def norm(lib, **kw):
    a = dict(x=FAKE, res=FAKE, dt=2, rows=4, cols=64, w=FAKE, wd=2, eps=1e-6, q=3, y=FAKE, h=FAKE, rstd=FAKE, codes=FAKE,
             scales=FAKE)
    a.update(kw)
    return lib.moe_rms_norm(a["x"], a["res"], a["dt"], a["rows"], a["cols"], a["w"], a["wd"], a["eps"], a["q"], a["y"],
                            a["h"], a["rstd"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(rows=1 << 24), 2), (dict(cols=0), 2), (dict(cols=16416), 2), (dict(cols=48), 2),
    (dict(dt=3), 3), (dict(dt=-1), 3), (dict(wd=1), 3), (dict(dt=0), 3), (dict(eps=0.0), 1), (dict(eps=-1e-6), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(q=1), 4), (dict(q=16), 4), (dict(x=None), 1),
    (dict(w=None), 1), (dict(rstd=None), 1), (dict(h=None), 1), (dict(codes=None), 1), (dict(scales=None), 1),
    (dict(q=-1, y=None), 1), (dict(x=FAKE + 1), 1), (dict(res=FAKE + 1), 1), (dict(codes=FAKE + 4), 1),
    (dict(rstd=FAKE + 2), 1), (dict(wd=0, w=FAKE + 2), 1), (dict(y=FAKE + 1), 1), (dict(h=FAKE + 1), 1),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status and lib.moe_last_error().decode()


def norm_back(lib, **kw):
    a = dict(g=FAKE, h=FAKE, gh=FAKE, dt=2, rows=4, cols=65, w=FAKE, wd=0, rstd=FAKE, gx=FAKE, gw=FAKE, work=FAKE,
             work_bytes=1 << 30)
    a.update(kw)
    return lib.moe_rms_norm_backward(a["g"], a["h"], a["gh"], a["dt"], a["rows"], a["cols"], a["w"], a["wd"], a["rstd"],
                                     a["gx"], a["gw"], a["work"], a["work_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(rows=1 << 24), 2), (dict(cols=0), 2), (dict(cols=16385), 2), (dict(dt=5), 3),
    (dict(wd=1), 3), (dict(g=None), 1), (dict(h=None), 1), (dict(w=None), 1), (dict(rstd=None), 1), (dict(gx=None), 1),
    (dict(gw=None), 1), (dict(g=FAKE + 1), 1), (dict(gh=FAKE + 1), 1), (dict(gx=FAKE + 1), 1), (dict(w=FAKE + 2), 1),
    (dict(gw=FAKE + 2), 1), (dict(work_bytes=0), 5), (dict(work=None), 5), (dict(work=FAKE + 16), 5),
])
def test_norm_backward_refusals(lib, kw, status):
    assert norm_back(lib, **kw) == status and lib.moe_last_error().decode()


def product(lib, **kw):
    a = dict(x=FAKE, dt=2, rows=64, off=FAKE, groups=4, w=FAKE, t=0, n=64, k=256, out=FAKE, od=2, work=FAKE,
             work_bytes=1 << 40)
    a.update(kw)
    return lib.moe_grouped_matmul(a["x"], a["dt"], a["rows"], a["off"], a["groups"], a["w"], a["t"], a["n"], a["k"],
                                  a["out"], a["od"], a["work"], a["work_bytes"], None)


def wgrad(lib, **kw):
    a = dict(g=FAKE, x=FAKE, dt=2, rows=64, off=FAKE, groups=4, n=64, k=256, out=FAKE, od=2, work=FAKE,
             work_bytes=1 << 40)
    a.update({{"w": "g"}.get(k, k): v for k, v in kw.items()})
    return lib.moe_grouped_matmul_wgrad(a["g"], a["x"], a["dt"], a["rows"], a["off"], a["groups"], a["n"], a["k"],
                                        a["out"], a["od"], a["work"], a["work_bytes"], None)


REFUSED = [
    (dict(rows=-1), 2), (dict(rows=1 << 24), 2), (dict(groups=0), 2), (dict(groups=1025), 2), (dict(n=0), 2),
    (dict(n=(1 << 20) + 1), 2), (dict(k=0), 2), (dict(k=(1 << 20) + 1), 2), (dict(dt=0), 3), (dict(dt=7), 3),
    (dict(od=1), 3), (dict(dt=1), 3), (dict(off=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1),
    (dict(x=FAKE + 1), 1), (dict(w=FAKE + 1), 1), (dict(out=FAKE + 1), 1), (dict(od=0, out=FAKE + 2), 1),
    (dict(off=FAKE + 2), 1),
]


@pytest.mark.parametrize("kw,status", REFUSED + [(dict(t=2), 1), (dict(t=-1), 1)])
def test_product_refusals(lib, kw, status):
    assert product(lib, **kw) == status and lib.moe_last_error().decode()


@pytest.mark.parametrize("kw,status", REFUSED)
def test_wgrad_refusals(lib, kw, status):
    assert wgrad(lib, **kw) == status and lib.moe_last_error().decode()


def test_workspaces(lib):
    b = ctypes.c_size_t()
    assert lib.moe_rms_norm_backward_workspace_size(8192, 7168, ctypes.byref(b)) == 0 and b.value >= 7168 * 4
    assert lib.moe_rms_norm_backward_workspace_size(8192, 0, ctypes.byref(b)) == 2
    assert lib.moe_rms_norm_backward_workspace_size(8192, 64, None) == 1
    for n, k in [(64, 64), (4096, 7168), (61, 33)]:
        for rows, groups in [(0, 1), (1, 8), (100, 8), (32768, 16)]:
            assert lib.moe_grouped_matmul_workspace_size(rows, groups, n, k, 1, ctypes.byref(b)) == 0
            if b.value and rows:   # without it the call is refused, naming the bytes
                assert product(lib, rows=rows, groups=groups, n=n, k=k, t=1, work_bytes=b.value - 1) == 5
                assert "bytes required" in lib.moe_last_error().decode()
            assert lib.moe_grouped_matmul_wgrad_workspace_size(rows, groups, n, k, ctypes.byref(b)) == 0
            if b.value:
                assert wgrad(lib, rows=rows, groups=groups, n=n, k=k, work_bytes=b.value - 1) == 5
    assert lib.moe_grouped_matmul_workspace_size(1, 1, 0, 4, 0, ctypes.byref(b)) == 2
    assert lib.moe_grouped_matmul_workspace_size(1, 1, 4, 4, 2, ctypes.byref(b)) == 1
    assert lib.moe_grouped_matmul_workspace_size(1, 1, 4, 4, 0, None) == 1
    assert lib.moe_grouped_matmul_wgrad_workspace_size(1, 1, 4, 4, None) == 1


def test_an_output_that_overlaps_an_operand_is_refused(lib):
    """Small and large forms, the output at, in front of and behind an operand's first byte."""
    for rows, n, k in ((4, 64, 256), (640, 64, 256)):
        apart = dict(x=FAKE << 20, w=FAKE << 21, out=FAKE << 22)
        for at in (apart["x"], apart["x"] + 2 * rows * k - 2, apart["x"] - 2 * rows * n + 2, apart["w"], apart["w"] + 2 * 4 * n * k - 2):
            assert product(lib, **{**apart, "rows": rows, "n": n, "k": k, "out": at}) == 1
            assert "overlaps" in lib.moe_last_error().decode()
        for at in (apart["x"], apart["x"] + 2 * rows * n - 2, apart["w"], apart["w"] - 2 * 4 * n * k + 2):
            assert wgrad(lib, **{**apart, "rows": rows, "n": n, "k": k, "out": at}) == 1
            assert "overlaps" in lib.moe_last_error().decode()


def test_planning_takes_no_time(lib):
    """The choice of a tile is not slower for more rows: the most rows, and every number of groups up to 8."""
    b, took = ctypes.c_size_t(), []
    for _ in range(3):
        t = time.perf_counter()
        for groups in range(1, 9):
            for trans in (0, 1):
                assert lib.moe_grouped_matmul_workspace_size((1 << 24) - 2, groups, 4096, 7168, trans, ctypes.byref(b)) == 0
        took.append(time.perf_counter() - t)
    assert min(took) < 0.02   # (a sum over all tiles would take 0.3 s)


def test_nothing_to_do_launches_nothing(lib):
    assert norm(lib, rows=0, x=None, w=None, y=None, h=None, rstd=None, codes=None, scales=None) == 0
    assert product(lib, rows=0, x=None, w=None, out=None) == 0


def test_norm_binding_refusals():
    """Shapes and types the library would misread are refused before any call (on the host)."""
    x, w = torch.zeros((4, 64)), torch.zeros(64)
    bad = [((x.double(), w), {}), ((x[0], w), {}), ((x, w[:63]), {}), ((x, w.half()), {}), ((x.half(), w.bfloat16()), {}),
           ((x, w, x.half()), {}), ((x, w, x[:3]), {}), ((x, w), dict(want_y=False)), ((x, w), {})]   # the last: not on the GPU
    for args, kw in bad:
        with pytest.raises(ValueError):
            rp.rms_norm(*args, **kw)
    r = torch.zeros(4)
    bad = [((x, x.half(), w, r), {}), ((x[:3], x, w, r), {}), ((x, x, w[:1], r), {}), ((x, x, w, r[:3]), {}),
           ((x, x, w, r.double()), {}), ((x, x, w, r), dict(grad_h=x[:, :32])), ((x, x, w, r), {})]
    for args, kw in bad:
        with pytest.raises(ValueError):
            rp.rms_norm_backward(*args, **kw)


def test_product_binding_refusals():
    x, w = torch.zeros((6, 32), dtype=torch.float16), torch.zeros((2, 16, 32), dtype=torch.float16)
    off = torch.zeros(3, dtype=torch.int32)
    good = dict(group_offsets=off)
    bad = [((x.float(), w), good), ((x, w.bfloat16()), good), ((x, w), {}), ((x[:, :31], w), good), ((x, w), dict(good, transpose_w=True)),
           ((x, w[0]), good), ((x[0], w), good), ((x, w), dict(group_offsets=off.long())), ((x, w), dict(group_offsets=off[:2])),
           ((x, w), dict(group_offsets=off[None])), ((x, w), dict(good, out_dtype=torch.bfloat16)),
           ((x, w), dict(good, out=torch.zeros((6, 15), dtype=torch.float16))),
           ((x, w), dict(good, out=torch.zeros((6, 16), dtype=torch.bfloat16))),
           ((x, w), dict(good, out=torch.zeros((6, 16)), out_dtype=torch.float16)),
           ((x, w), dict(good, workspace=torch.zeros(8))), ((x, w), good)]   # the last: not on the GPU
    for args, kw in bad:
        with pytest.raises(ValueError):
            rp.grouped_matmul(*args, **kw)
    g = torch.zeros((6, 16), dtype=torch.float16)
    bad = [((g.float(), x), good), ((g[:5], x), good), ((g, x.float()), good), ((g, x), dict(group_offsets=off.long())),
           ((g, x), dict(good, out_dtype=torch.bfloat16)), ((g, x), dict(good, out=torch.zeros((16, 32)))),
           ((g, x), dict(out=torch.zeros((1, 16, 32)))), ((g, x), dict(good, workspace=torch.zeros(8))), ((g, x), good)]
    for args, kw in bad:
        with pytest.raises(ValueError):
            rp.grouped_matmul_wgrad(*args, **kw)
