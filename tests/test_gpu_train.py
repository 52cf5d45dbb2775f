"""One run of the operators as a training step of a layer uses them: norm of the residual stream ->
router's product -> gate_topk -> token_permute -> expert products (torch's SwiGLU between) ->
weighted sum, and the way back through gate_backward, the products' and the norm's gradients; the
gradients against float64 autograd of the same layer with the choice of experts held fixed. And the
norm's codes as the input of an MXFP8 layer."""
import pytest
import torch

import moe_inputs
import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, FP8, oracle_weights, to_dev

pytestmark = pytest.mark.gpu


def test_training_step():
    n, c, e, k, inter = 200, 512, 8, 2, 192
    gen = torch.Generator().manual_seed(0)
    draw = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, res, wn = draw(n, c), draw(n, c, std=2.0), 1 + draw(c, std=0.2)
    wr, w1, w2 = draw(e, c, std=c ** -0.5), draw(e, 2 * inter, c, std=c ** -0.5), draw(e, c, inter, std=inter ** -0.5)
    g = draw(n, c, std=0.1)

    # forward
    y, h, rstd, _, _ = rp.rms_norm(x, wn, res)
    logits = rp.grouped_matmul(y, wr, out_dtype=torch.float32)
    ids, weights = rp.gate_topk(logits, k)
    rows, index, _ = rp.token_permute(y, ids, num_experts=e)
    index = index.long()   # sorted place of each (token, choice)
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.bincount(ids.reshape(-1).long(), minlength=e).cumsum(0)])
    off = off.to(torch.int32)
    z = rp.grouped_matmul(rows, w1, off)
    za = z.float().requires_grad_(True)
    act = torch.nn.functional.silu(za[:, :inter]) * za[:, inter:]
    a = act.to(torch.bfloat16).detach()
    o = rp.grouped_matmul(a, w2, off)
    out = h.float() + (o.float()[index].view(n, k, c) * weights[:, :, None]).sum(1)

    # back
    chosen = o.float()[index].view(n, k, c)
    gw_gate = (chosen * g.float()[:, None]).sum(2)
    go = torch.empty_like(o)
    go[index] = (g.float()[:, None] * weights[:, :, None]).reshape(n * k, c).to(torch.bfloat16)
    gw2 = rp.grouped_matmul_wgrad(go, a, off, out_dtype=torch.float32)
    ga = rp.grouped_matmul(go, w2, off, transpose_w=True, out_dtype=torch.float32)
    gz, = torch.autograd.grad(act, za, ga)
    gz = gz.to(torch.bfloat16)
    gw1 = rp.grouped_matmul_wgrad(gz, rows, off, out_dtype=torch.float32)
    grows = rp.grouped_matmul(gz, w1, off, transpose_w=True, out_dtype=torch.float32)
    glog = rp.gate_backward(logits, ids, gw_gate)
    glog16 = glog.to(torch.bfloat16)
    gwr = rp.grouped_matmul_wgrad(glog16, y, out_dtype=torch.float32)
    gy = grows[index].view(n, k, c).sum(1) + rp.grouped_matmul(glog16, wr, transpose_w=True, out_dtype=torch.float32)
    gx, gwn = rp.rms_norm_backward(gy.to(torch.bfloat16), h, wn, rstd, grad_h=g)

    # float64, the same choice
    d = [t.double().requires_grad_(True) for t in (x, res, wn, wr, w1, w2)]
    dx, dres, dwn, dwr, dw1, dw2 = d
    hh = dx + dres
    yy = hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + 1e-6) * dwn
    p = torch.softmax(yy @ dwr.T, 1).gather(1, ids.long())
    p = p / p.sum(1, keepdim=True)
    total = hh
    for j in range(k):
        zz = torch.einsum("nc,nic->ni", yy, dw1[ids[:, j].long()])
        aa = torch.nn.functional.silu(zz[:, :inter]) * zz[:, inter:]
        total = total + p[:, j:j + 1] * torch.einsum("ni,nci->nc", aa, dw2[ids[:, j].long()])
    want = torch.autograd.grad((total * g.double()).sum(), d)
    # Each of at most 12 roundings to bf16 between the input and a result is off by at most 2^-8 of
    # its value; they add up at random over the sums (c, inter or n terms), so that the whole differs by
    # no more than 12 2^-8 / sqrt(3) of its norm (uniform errors), about 2.7e-2; the products' own
    # errors (1e-6) vanish beside it.
    def near(got, ref):
        return float((got.double() - ref).norm() / ref.norm()) < 2.7e-2

    assert near(out, total.detach())
    for name, got, ref in (("x", gx, want[0]), ("residual", gx, want[1]), ("norm weight", gwn, want[2]),
                           ("router", gwr, want[3]), ("w1", gw1, want[4]), ("w2", gw2, want[5])):
        assert near(got, ref), name


def test_codes_as_the_layers_input():
    """rms_norm's MXFP8 codes and scales through mega_moe: the same bits as its y quantised by the layer."""
    cfg = moe_inputs.config("tiny")
    x = moe_inputs.activations(cfg).to(DEV)
    w = torch.ones(cfg.hidden, dtype=torch.bfloat16, device=DEV)
    ids, tw = to_dev(moe_inputs.expert_ids(cfg)), to_dev(moe_inputs.gate_weights(cfg))
    weights = [to_dev(a) for a in oracle_weights(cfg)]
    y, _, _, codes, scales = rp.rms_norm(x, w, x, quant_mode=rp.QUANT_E4M3)
    direct, _ = rp.mega_moe(y, ids, tw, *weights, quant_out_dtype=FP8["e4m3"])
    coded, _ = rp.mega_moe(codes, ids, tw, *weights, quant_out_dtype=FP8["e4m3"], x_scales=scales)
    assert torch.equal(direct, coded)
