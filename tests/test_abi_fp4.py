"""Host-side refusals of the MXFP4 product: wrong arguments return an error with a message
before any launch, so these run without a GPU."""
import ctypes
import os

import pytest
import torch

import routing_permute_mxfp8_amd as rp

FAKE = 0x1000   # never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rp.lib_path()):
        from routing_permute_mxfp8_amd import build
        build.build()
    return rp.load()


def call(lib, **kw):
    a = dict(x=FAKE, xd=2, xs=None, rows=64, off=FAKE, groups=4, w=FAKE, ws=FAKE, n=64, k=256, fmt=0, out=FAKE, od=2,
             work=None, work_bytes=0)
    a.update(kw)
    return lib.moe_mxfp4_matmul(a["x"], a["xd"], a["xs"], a["rows"], a["off"], a["groups"], a["w"], a["ws"], a["n"],
                                a["k"], a["fmt"], a["out"], a["od"], a["work"], a["work_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(rows=1 << 24), 2), (dict(groups=0), 2), (dict(groups=1025), 2), (dict(n=0), 2),
    (dict(n=24), 2), (dict(n=(1 << 20) + 16), 2), (dict(k=0), 2), (dict(k=192), 2), (dict(k=65536 + 128), 2),
    (dict(xd=3), 3), (dict(xd=5), 3), (dict(fmt=2), 1), (dict(od=1), 3), (dict(off=None), 1), (dict(x=None), 1),
    (dict(w=None), 1), (dict(ws=None), 1), (dict(out=None), 1), (dict(xs=FAKE), 1), (dict(xd=7), 1),
    (dict(x=FAKE + 8), 1), (dict(w=FAKE + 4), 1), (dict(out=FAKE + 2), 1), (dict(ws=FAKE + 2), 1),
    (dict(ws=FAKE + 4, fmt=1), 1), (dict(xd=7, xs=FAKE + 1), 1),
])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status and lib.moe_last_error().decode()


def test_workspace(lib):
    b = ctypes.c_size_t()
    assert lib.moe_mxfp4_matmul_workspace_size(1, 1, 64, 256, 2, 0, ctypes.byref(b)) == 0
    assert lib.moe_mxfp4_matmul_workspace_size(0, 8, 64, 256, 7, 1, ctypes.byref(b)) == 0
    assert lib.moe_mxfp4_matmul_workspace_size(1, 1, 64, 100, 2, 0, ctypes.byref(b)) == 2
    assert lib.moe_mxfp4_matmul_workspace_size(1, 1, 64, 256, 2, 0, None) == 1
    assert lib.moe_mxfp4_matmul_workspace_size(1 << 20, 1024, 8192, 8192, 0, 0, ctypes.byref(b)) == 0
    if b.value:   # a call of that size without it is refused, naming the bytes
        assert call(lib, rows=1 << 20, groups=1024, n=8192, k=8192, xd=0) == 5
        assert "bytes required" in lib.moe_last_error().decode()


def test_nothing_to_do_launches_nothing(lib):
    assert call(lib, rows=0, x=None, w=None, ws=None, out=None) == 0


def test_binding_refusals():
    """Shapes and types the library would misread are refused before any call (on the host)."""
    w = torch.zeros((2, 32, 64), dtype=torch.uint8)
    s = torch.zeros((2, 32, 4), dtype=torch.uint8)
    x = torch.zeros((6, 128))
    codes, cs = torch.zeros((6, 64), dtype=torch.uint8), torch.zeros((6, 4), dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    good = dict(group_offsets=off)
    bad = [((x, w, s), {}), ((x[:, :64], w, s), good), ((x.double(), w, s), good), ((codes, w, s), good),
           ((x, w, s), dict(good, x_scales=cs)), ((codes, w, s), dict(good, x_scales=cs[:, :3])),
           ((codes.to(torch.int8), w, s), dict(good, x_scales=cs)), ((x, w, s[:1]), good), ((x, w[:, :, 0], s), good),
           ((x, w, s), dict(group_offsets=off.long())), ((x, w, s), dict(group_offsets=off[:2])),
           ((x, w, s), dict(good, out_dtype=torch.float16)), ((x, w, s), dict(good, out=torch.zeros((6, 31)))),
           ((x, w, s), dict(good, out=torch.zeros((6, 32), dtype=torch.float16))),
           ((x, w, s), dict(good, weight_format=rp.WEIGHTS_PACKED)),
           ((x, w, s), dict(good, workspace=torch.zeros(8))), ((x, w, s), good)]   # the last: not on the GPU
    for args, kw in bad:
        with pytest.raises(ValueError):
            rp.mxfp4_matmul(*args, **kw)
