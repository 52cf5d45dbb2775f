"""Host-side refusals of the router's entry points: wrong arguments return an error with a
message before any launch, so these run without a GPU."""
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


def gate(lib, **kw):
    a = dict(logits=FAKE, dtype=0, rows=4, e=256, k=8, scoring=0, bias=None, groups=8, keep=4, renorm=1, scale=1.0,
             ids=FAKE, w=FAKE)
    a.update(kw)
    return lib.moe_gate_topk(a["logits"], a["dtype"], a["rows"], a["e"], a["k"], a["scoring"], a["bias"], a["groups"],
                             a["keep"], a["renorm"], a["scale"], a["ids"], a["w"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(rows=1 << 31), 2), (dict(e=0), 2), (dict(e=1025, groups=1, keep=1), 2), (dict(k=0), 2),
    (dict(k=33), 2), (dict(e=4, groups=1, keep=1), 2), (dict(dtype=3), 3), (dict(scoring=2), 1), (dict(groups=0), 2),
    (dict(groups=3), 2), (dict(groups=128), 2), (dict(keep=0), 2), (dict(keep=9), 2), (dict(k=32, e=64, keep=3), 2),
    (dict(renorm=2), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(logits=None), 1),
    (dict(ids=None), 1), (dict(w=None), 1),
])
def test_gate_topk_refusals(lib, kw, status):
    assert gate(lib, **kw) == status and lib.moe_last_error().decode()


def test_gate_topk_without_rows_launches_nothing(lib):
    assert gate(lib, rows=0, logits=None, ids=None, w=None) == 0


def balance(lib, **kw):
    a = dict(logits=FAKE, dtype=0, rows=4, e=256, ids=FAKE, k=8, scoring=0, off=FAKE, seqs=2, mask=None, alpha=1.0,
             loss=FAKE, counts=FAKE, coef=FAKE, ws=FAKE, ws_bytes=0)
    a.update(kw)
    return lib.moe_balance_loss(a["logits"], a["dtype"], a["rows"], a["e"], a["ids"], a["k"], a["scoring"], a["off"],
                                a["seqs"], a["mask"], a["alpha"], a["loss"], a["counts"], a["coef"], a["ws"],
                                a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(e=2000), 2), (dict(k=33), 2), (dict(dtype=4), 3), (dict(scoring=-1), 1),
    (dict(seqs=0), 2), (dict(seqs=65536), 2), (dict(off=None), 1), (dict(alpha=float("nan")), 1),
    (dict(logits=None), 1), (dict(ids=None), 1), (dict(loss=None), 1), (dict(counts=None), 1), (dict(coef=None), 1),
    (dict(), 5), (dict(ws=None, ws_bytes=1 << 30), 5), (dict(ws=0x1001, ws_bytes=1 << 30), 5),
])
def test_balance_loss_refusals(lib, kw, status):
    assert balance(lib, **kw) == status
    msg = lib.moe_last_error().decode()
    assert msg and (status != 5 or "bytes required" in msg or "aligned" in msg)


def test_balance_loss_workspace(lib):
    b = ctypes.c_size_t()
    assert lib.moe_balance_loss_workspace_size(32768, 256, 8, ctypes.byref(b)) == 0
    assert 0 < b.value < 8 << 20
    assert lib.moe_balance_loss_workspace_size(1 << 30, 1024, 65535, ctypes.byref(b)) == 0 and b.value > 0
    assert lib.moe_balance_loss_workspace_size(8, 0, 1, ctypes.byref(b)) == 2
    assert lib.moe_balance_loss_workspace_size(8, 8, 0, ctypes.byref(b)) == 2
    assert lib.moe_balance_loss_workspace_size(8, 8, 1, None) == 1


def backward(lib, **kw):
    a = dict(logits=FAKE, dtype=0, rows=4, e=256, ids=FAKE, k=8, scoring=0, renorm=1, scale=1.0, gw=FAKE, gl=FAKE,
             coef=FAKE, off=FAKE, seqs=2, mask=None, grad=FAKE)
    a.update(kw)
    return lib.moe_gate_backward(a["logits"], a["dtype"], a["rows"], a["e"], a["ids"], a["k"], a["scoring"],
                                 a["renorm"], a["scale"], a["gw"], a["gl"], a["coef"], a["off"], a["seqs"], a["mask"],
                                 a["grad"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 2), (dict(e=2000), 2), (dict(k=0), 2), (dict(dtype=5), 3), (dict(scoring=7), 1),
    (dict(seqs=0), 2), (dict(off=None), 1), (dict(renorm=-1), 1), (dict(scale=float("inf")), 1), (dict(coef=None), 1),
    (dict(gl=None), 1), (dict(gw=None, gl=None, coef=None), 1), (dict(logits=None), 1), (dict(ids=None), 1),
    (dict(grad=None), 1),
])
def test_gate_backward_refusals(lib, kw, status):
    assert backward(lib, **kw) == status and lib.moe_last_error().decode()


def test_binding_refusals():
    """Shapes and types the library would misread are refused before any call (on the host)."""
    x = torch.zeros((4, 8))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    w = torch.zeros((4, 2))
    for bad in (x.double(), x[0], x.to(torch.int32)):
        with pytest.raises(ValueError):
            rp.gate_topk(bad, 2)
    with pytest.raises(ValueError):   # not on the GPU
        rp.gate_topk(x, 2)
    for bad in (ids.long(), ids[:3], ids[:, 0]):
        with pytest.raises(ValueError):
            rp.balance_loss(x, bad)
        with pytest.raises(ValueError):
            rp.gate_backward(x, bad, w)
    for kw in (dict(seq_offsets=torch.zeros(3, dtype=torch.int64)), dict(seq_offsets=torch.zeros(1, dtype=torch.int32)),
               dict(row_mask=torch.ones(3, dtype=torch.uint8)), dict(row_mask=torch.ones(4))):
        with pytest.raises(ValueError):
            rp.balance_loss(x, ids, **kw)
        with pytest.raises(ValueError):
            rp.gate_backward(x, ids, w, **kw)
    for kw in (dict(grad_weights=w.double()), dict(grad_weights=w[:, :1]), dict(grad_loss=torch.ones(2)),
               dict(coef=torch.ones(1, 9)), dict(coef=torch.ones(8))):
        with pytest.raises(ValueError):
            rp.gate_backward(x, ids, **kw)
