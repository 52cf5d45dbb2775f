"""The measured cases of the router and MXFP4 product operators: their inputs, plain forms, calls and exact values.

Four operators of an MoE layer, each in a plain torch form (own = False) and as the library's call (own = True):

  gate      topk_ids, topk_weights of rows of expert logits: softmax or sigmoid scores, a selection bias,
            group-limited selection, renormalised weights;
  balance   the load-balance loss of those rows over (ragged) sequences, with per-expert counts and the loss's
            derivative by each score;
  gradient  the logits' gradient from the gradients of the gate weights and of the balance loss;
  product   out = DQ(x) DQ(w_g)^T for the rows of each expert group, both operands MXFP4 (E2M1 codes two a byte,
            E8M0 scale per 32), x given as codes or quantised in the call.
"""

import math

import torch

own = False

DEV = "cuda"
FLOATS = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of one request: 256 experts in 8 groups, 4 of them allowed, bias-corrected sigmoid scores
        dict(name="gate 1x256 sigmoid groups", op="gate", rows=1, experts=256, k=8, scoring="sigmoid", dtype="fp32",
             bias=True, groups=8, topk_groups=4, renorm=True, scale=2.5, dead=0),
        # a prefill batch of the prefill workload (8192 tokens, 256 experts, topK 8), softmax scores
        dict(name="gate 8192x256 softmax", op="gate", rows=8192, experts=256, k=8, scoring="softmax", dtype="fp32",
             bias=False, groups=1, topk_groups=1, renorm=True, scale=1.0, dead=0),
        # the routing workload's batch (32768 tokens), bf16 logits straight from the gate's product
        dict(name="gate 32768x256 sigmoid groups", op="gate", rows=32768, experts=256, k=8, scoring="sigmoid",
             dtype="bf16", bias=True, groups=8, topk_groups=4, renorm=True, scale=2.5, dead=0),
        # a training step's balance loss, one loss for each of 8 sequences of different lengths
        dict(name="balance 32768x256 ragged", op="balance", rows=32768, experts=256, k=8, scoring="softmax",
             dtype="fp32", seqs=8, masked=False, alpha=0.01),
        # a small padded batch of a layer with an odd number of experts: masked rows do not count
        dict(name="balance 1000x60 masked", op="balance", rows=1000, experts=60, k=4, scoring="sigmoid", dtype="fp32",
             seqs=1, masked=True, alpha=0.001),
        # the backward pass of the training step above: gate weights and balance loss at once
        dict(name="gradient 32768x256 ragged", op="gradient", rows=32768, experts=256, k=8, scoring="softmax",
             dtype="fp32", seqs=8, masked=False, alpha=0.01, renorm=True, scale=1.0),
        # the backward pass of a small odd layer: bf16 logits, sigmoid scores, padded rows
        dict(name="gradient 517x60 masked", op="gradient", rows=517, experts=60, k=4, scoring="sigmoid", dtype="bf16",
             seqs=3, masked=True, alpha=0.001, renorm=True, scale=2.5),
        # a dense projection of one token (hidden 7168 to 2 x 2048 channels), bf16 x quantised in the call
        dict(name="product 1 row dense", op="product", rows=1, groups=1, k=7168, n=4096, x="bf16", out="bf16", skew=0.0),
        # decode of the decode workload on a quarter of its experts: 128 tokens x topK 8 / 4 = 256 rows on 64 experts
        dict(name="product 256 rows 64 experts", op="product", rows=256, groups=64, k=7168, n=4096, x="codes",
             out="bf16", skew=0.0),
        # the up projection of a large prefill batch, 2048 rows an expert
        dict(name="product 32768 rows 16 experts", op="product", rows=32768, groups=16, k=7168, n=4096, x="codes",
             out="bf16", skew=0.0),
        # the down projection of a prefill batch (inter 2048 to hidden 7168), 256 rows an expert, bf16 activations
        dict(name="product 8192 rows down", op="product", rows=8192, groups=32, k=2048, n=7168, x="bf16", out="bf16",
             skew=0.0),
        # a ragged batch: odd row count, experts without rows, sizes that fill no tile, fp32 sums for a later reduction
        dict(name="product 777 rows ragged", op="product", rows=777, groups=5, k=1408, n=2000, x="fp16", out="fp32",
             skew=1.0),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "balance", "gradient", "product", "product"])
    if op == "product":
        while True:
            c = dict(op=op, rows=_between(rng, 1, 32768), groups=_between(rng, 1, 64), k=128 * _between(rng, 1, 64),
                     n=16 * _between(rng, 4, 512), x=rng.choice(["codes", "bf16", "fp16", "fp32"]),
                     out=rng.choice(["bf16", "fp32"]), skew=rng.choice([0.0, 0.0, 0.5, 1.0]))
            w, top = work(c), [work(d) for d in listed()]
            # a skewed batch's plain form pads every group to the longest
            padded = c["rows"] * (1.0 if c["skew"] == 0.0 or c["groups"] == 1 else c["groups"]) * (c["k"] + c["n"])
            if (w["flops"] <= max(t["flops"] for t in top) and w["bytes"] <= max(t["bytes"] for t in top)
                    and padded <= 5e8):
                return c
    experts = rng.choice([8, 16, 32, 60, 64, 72, 100, 128, 160, 256, 384, 512])
    k = rng.randint(1, min(experts, 10))
    c = dict(op=op, rows=_between(rng, 1, 32768 * 256 // max(experts, 256)), experts=experts, k=k,
             scoring=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16", "fp16"]))
    if op == "gate":
        groups = rng.choice([g for g in (1, 1, 2, 4, 8, 12) if experts % g == 0])
        most = -(-k * groups // experts)  # groups that hold k experts at least
        c.update(bias=rng.random() < 0.5, groups=groups, topk_groups=rng.randint(most, groups),
                 renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dead=rng.choice([0, 0, experts // 8]))
    else:
        c.update(seqs=min(c["rows"], rng.choice([1, 1, 3, 8, 31])), masked=rng.random() < 0.4,
                 alpha=rng.choice([0.01, 0.001]))
        if op == "gradient":
            c.update(renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    return c


def work(case):
    rows = case["rows"]
    if case["op"] == "product":
        groups, k, n = min(case["groups"], rows), case["k"], case["n"]
        xb = k * 17 / 32 if case["x"] == "codes" else k * SIZE[case["x"]]
        return dict(bytes=groups * n * k * 17 / 32 + rows * (xb + n * SIZE[case["out"]]), flops=2.0 * rows * n * k)
    e, k, sz = case["experts"], case["k"], SIZE[case["dtype"]]
    if case["op"] == "gate":  # logits in, ids and weights out; an exponential, its sum and a comparison each
        return dict(bytes=rows * (e * sz + 8 * k) + (4 * e if case["bias"] else 0), flops=rows * e * 8.0)
    if case["op"] == "balance":  # logits and ids in; counts and derivatives out
        return dict(bytes=rows * (e * sz + 4 * k) + case["seqs"] * e * 8 + 4, flops=rows * e * 8.0)
    # logits, ids, weight gradients in; logit gradients out
    return dict(bytes=rows * (2 * e * sz + 8 * k) + case["seqs"] * e * 4, flops=rows * e * 12.0)


# ---- inputs --------------------------------------------------------------------------------------------------------
def _codes(x):
    """MXFP4 codes [..., K/2] and E8M0 scales [..., K/32] of x (fp32): what a user keeps of quantised weights or rows."""
    v, b = _mx_parts(x)
    mag = v.abs()
    code = sum((mag >= t).to(torch.uint8) for t in E2M1[1:])
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), b.reshape(*x.shape[:-1], x.shape[-1] // 32)


def _sizes(case, gen):
    """Rows of each group on the host: drawn uniformly, or with p(rank) ~ rank^-skew and the second group empty."""
    groups = case["groups"]
    p = torch.arange(1, groups + 1, dtype=torch.float64) ** -case["skew"]
    if case["skew"] > 0 and groups > 2:
        p[1] = 0.0
    got = torch.multinomial(p / p.sum(), case["rows"], replacement=True, generator=gen)
    return torch.bincount(got, minlength=groups)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    rows = case["rows"]
    s = dict(case=case)
    if case["op"] == "product":
        groups, n, k = case["groups"], case["n"], case["k"]
        s["w"] = torch.empty((groups, n, k // 2), dtype=torch.uint8, device=DEV)
        s["ws"] = torch.empty((groups, n, k // 32), dtype=torch.uint8, device=DEV)
        for g in range(0, groups, 4):  # a few experts' float weights at a time
            m = torch.randn((min(4, groups - g), n, k), generator=gen, device=DEV) / math.sqrt(k)
            s["w"][g:g + 4], s["ws"][g:g + 4] = _codes(m)
        x = torch.randn((rows, k), generator=gen, device=DEV)
        s["x"], s["xs"] = _codes(x) if case["x"] == "codes" else (x.to(FLOATS[case["x"]]), None)
        size = _sizes(case, host) if groups > 1 else torch.tensor([rows])
        end = torch.cumsum(size, 0)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), end]).to(torch.int32).to(DEV)
        # the plain form's padding: row of each slot of [groups, longest], slot of each row
        longest = int(size.max())
        slot = (end - size)[:, None] + torch.arange(longest)
        group = torch.repeat_interleave(torch.arange(groups), size)
        s["slot"] = slot.clamp(max=rows - 1).to(DEV)
        s["place"] = (group * longest + torch.arange(rows) - (end - size)[group]).to(DEV)
        return s
    e, k = case["experts"], case["k"]
    logits = torch.randn((rows, e), generator=gen, device=DEV) * 1.5
    if case["op"] == "gate":
        if case["dead"]:  # experts taken out of service
            logits[:, torch.randperm(e, generator=host)[:min(case["dead"], e - k)].to(DEV)] = -math.inf
        s["logits"] = logits.to(FLOATS[case["dtype"]])
        # a bias learned to even out the load: small beside the scores
        s["bias"] = torch.randn((e,), generator=gen, device=DEV) * 0.05 if case["bias"] else None
        return s
    s["logits"] = logits.to(FLOATS[case["dtype"]])
    s["ids"] = s["logits"].float().topk(k, dim=1).indices.to(torch.int32)
    cut = torch.randperm(rows - 1, generator=host)[:case["seqs"] - 1].sort().values + 1 if case["seqs"] > 1 else []
    s["offsets"] = torch.tensor([0, *[int(c) for c in cut], rows], dtype=torch.int32, device=DEV)
    s["mask"] = (torch.rand((rows,), generator=gen, device=DEV) < 0.8).to(torch.uint8) if case["masked"] else None
    if case["op"] == "gradient":
        s["gw"] = torch.randn((rows, k), generator=gen, device=DEV) * 0.1
        s["gl"] = torch.rand((1,), generator=gen, device=DEV) + 0.5
        # kept from the forward pass: the loss's derivative by each score of a counted row
        s["coef"] = _balance(s["logits"], s["ids"], s["offsets"], s["mask"], case)[2]
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------------
def _mx_parts(x):
    """x (fp32) as E2M1 values of its 32-groups and their E8M0 bytes: shared exponent floor(log2 amax) - 2, elements
    rounded to the nearest of E2M1 (ties to the even code), magnitudes above 6 held at 6."""
    v = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = v.abs().amax(-1, keepdim=True)
    b = (torch.frexp(amax).exponent + 124).clamp(0, 254)  # frexp: amax = m 2^e, m in [0.5, 1)
    b = torch.where(amax > 0, b, 0)
    v = torch.ldexp(v, 127 - b)
    a = v.abs()
    r = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0)
    return torch.copysign(r, v).reshape(x.shape), b.to(torch.uint8)


def _mx_values(codes, scales):
    """The fp32 values of MXFP4 codes [..., K/2] and scales [..., K/32]."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack([t.repeat(16), t.repeat_interleave(16)], 1)
    v = pair[codes.int()].reshape(*scales.shape, 32)
    v *= torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)[..., None]
    return v.reshape(*codes.shape[:-1], codes.shape[-1] * 2)


def _product(s):
    case = s["case"]
    if s["xs"] is None:
        v, b = _mx_parts(s["x"].float())
        x = torch.ldexp(v.reshape(*b.shape[:-1], 32), b.int() - 127).reshape(v.shape)
    else:
        x = _mx_values(s["x"], s["xs"])
    out = torch.bmm(x[s["slot"]], _mx_values(s["w"], s["ws"]).transpose(1, 2))
    return out.reshape(-1, case["n"])[s["place"]].to(FLOATS[case["out"]])


def _scores(logits, scoring, real):
    """Scores of logits in the type `real`: softmax or sigmoid; 0 where a logit is -inf, and in a row of them."""
    x = logits.to(real)
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=torch.finfo(real).min))
    return e / e.sum(1, keepdim=True).clamp(min=torch.finfo(real).tiny)


def _gate(s):
    case, logits = s["case"], s["logits"]
    rows, e = logits.shape
    live = logits > -math.inf
    if s["bias"] is None and case["groups"] == 1:
        rank = logits.double()  # the scores rise with the logits
    else:  # in 64 bits: two scores may lie next to each other
        rank = _scores(logits, case["scoring"], torch.float64)
        rank = rank + s["bias"].double() if s["bias"] is not None else rank
        rank = torch.where(live, rank, -1e30)
    if case["groups"] > 1:
        two = rank.reshape(rows, case["groups"], -1)
        two = two.sort(dim=2, descending=True).values[:, :, :2]
        second = torch.where(two[:, :, 1] > -1e30, two[:, :, 1], 0.0) if two.shape[2] > 1 else 0.0
        order = (two[:, :, 0] + second).sort(dim=1, descending=True, stable=True).indices
        allowed = torch.zeros((rows, case["groups"]), dtype=torch.bool, device=logits.device)
        allowed.scatter_(1, order[:, :case["topk_groups"]], True)
        rank = torch.where(allowed.repeat_interleave(e // case["groups"], 1), rank, -math.inf)
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]
    w = _scores(logits, case["scoring"], torch.float32).gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
    return ids.to(torch.int32), w * case["scale"]


def _probabilities(logits, scoring):
    p = _scores(logits, scoring, torch.float32)
    return p / p.sum(1, keepdim=True) if scoring == "sigmoid" else p


def _segments(offsets, mask, rows):
    """Sequence of each row, and 1 where the row counts."""
    at = torch.arange(rows, device=offsets.device)
    seq = torch.bucketize(at, offsets[1:].long(), right=True)
    counted = torch.ones((rows,), device=offsets.device) if mask is None else (mask != 0).float()
    return seq, counted


def _balance(logits, ids, offsets, mask, case):
    rows, e = logits.shape
    seqs = offsets.numel() - 1
    seq, counted = _segments(offsets, mask, rows)
    # sums over each sequence as differences of running sums along the rows, in 64 bits
    chosen = torch.zeros((rows, e), device=logits.device).scatter_(1, ids.long(), 1.0)
    terms = torch.cat([_probabilities(logits, case["scoring"]), chosen, torch.ones_like(counted)[:, None]], 1)
    running = torch.zeros((2 * e + 1, rows + 1), dtype=torch.float64, device=logits.device)
    torch.cumsum((terms * counted[:, None]).T.contiguous(), 1, dtype=torch.float64, out=running[:, 1:])
    sums, counts, held = (running[:, offsets[1:].long()] - running[:, offsets[:-1].long()]).T.split([e, e, 1], 1)
    held = held[:, 0]
    filled = (held > 0).double().sum().clamp(min=1)
    coef = case["alpha"] * e / ids.shape[1] * counts / (held.clamp(min=1) ** 2)[:, None] / filled
    return (coef * sums).sum().reshape(1).float(), counts.to(torch.int32), coef.float()


def _gradient(s):
    case, logits, ids = s["case"], s["logits"], s["ids"].long()
    rows, e = logits.shape
    score = _scores(logits, case["scoring"], torch.float32)
    w = score.gather(1, ids)
    g = s["gw"] * case["scale"]
    if case["renorm"]:
        total = w.sum(1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)
        g = (g - (g * w / total).sum(1, keepdim=True)) / total
    dscore = torch.zeros((rows, e), device=logits.device).scatter_(1, ids, g)
    seq, counted = _segments(s["offsets"], s["mask"], rows)
    dp = s["coef"][seq] * (s["gl"] * counted)[:, None]
    if case["scoring"] == "softmax":
        d = dscore + dp
        d = score * (d - (d * score).sum(1, keepdim=True))
    else:
        z = score.sum(1, keepdim=True)
        d = dscore + (dp - (dp * score / z).sum(1, keepdim=True)) / z
        d = d * score * (1.0 - score)
    return d.to(logits.dtype)


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "product":
            return _product(s)
        if op == "gate":
            return _gate(s)
        if op == "balance":
            return _balance(s["logits"], s["ids"], s["offsets"], s["mask"], case)
        return _gradient(s)
    import routing_permute_mxfp8_amd as rp
    if op == "product":
        return rp.mxfp4_matmul(s["x"], s["w"], s["ws"], x_scales=s["xs"],
                               group_offsets=s["offsets"] if case["groups"] > 1 else None,
                               out_dtype=FLOATS[case["out"]])
    scoring = rp.GATE_SOFTMAX if case["scoring"] == "softmax" else rp.GATE_SIGMOID
    if op == "gate":
        return rp.gate_topk(s["logits"], case["k"], scoring=scoring, bias=s["bias"], num_groups=case["groups"],
                            topk_groups=case["topk_groups"], renormalize=case["renorm"], scale=case["scale"])
    if op == "balance":
        return rp.balance_loss(s["logits"], s["ids"], scoring=scoring, seq_offsets=s["offsets"], row_mask=s["mask"],
                               alpha=case["alpha"])
    return rp.gate_backward(s["logits"], s["ids"], s["gw"], scoring=scoring, renormalize=case["renorm"],
                            scale=case["scale"], grad_loss=s["gl"], coef=s["coef"].contiguous(), seq_offsets=s["offsets"],
                            row_mask=s["mask"])


# ---- from the definitions, in 64 bits ------------------------------------------------------------------------------
def _nearest(x):
    """x (64 bits) quantised to MXFP4 and back: the nearest of the eight magnitudes, looked for among the even codes
    first, of x over the power of two that brings its 32-group's largest magnitude into [4, 8)."""
    g = x.reshape(-1, 32)
    top = g.abs().max(1, keepdim=True).values
    step = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))).clamp(min=-125) - 2)
    mags = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=x.device)
    out = torch.empty_like(g)
    for part in range(0, g.shape[0], 1 << 20):
        y = g[part:part + (1 << 20)] / step[part:part + (1 << 20)]
        best = (y.abs()[..., None] - mags).abs().min(-1).indices
        out[part:part + (1 << 20)] = mags[best] * torch.sign(y) * step[part:part + (1 << 20)]
    return out.reshape(x.shape)


def _decoded(codes, scales):
    """MXFP4 codes in 64 bits from their sign, exponent and mantissa bits."""
    half = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    expo, man = ((half >> 1) & 3).double(), (half & 1).double()
    mag = torch.where(expo == 0, man / 2, (1 + man / 2) * torch.exp2(expo - 1))
    mag = torch.where(half > 7, -mag, mag)
    return mag * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        x = _nearest(s["x"].double()) if s["xs"] is None else _decoded(s["x"], s["xs"])
        out = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device=DEV)
        ends = s["offsets"].tolist()
        for g, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
            if hi > lo:
                out[lo:hi] = x[lo:hi] @ _decoded(s["w"][g], s["ws"][g]).T
        return out
    x = s["logits"].double()
    soft = case["scoring"] == "softmax"
    score = torch.softmax(x, 1) if soft else torch.sigmoid(x)
    if op == "gate":
        ids = _gate(s)[0]  # whole numbers have no error
        w = score.gather(1, ids.long())
        w = w / w.sum(1, keepdim=True) if case["renorm"] else w
        return None, w * case["scale"]
    # one sequence after the other, with autograd for the derivatives
    x.requires_grad_(True)
    score = torch.softmax(x, 1) if soft else torch.sigmoid(x)
    share = score if soft else score / score.sum(1, keepdim=True)
    ends, k, e = s["offsets"].tolist(), case["k"], case["experts"]
    keep = torch.ones((case["rows"],), device=DEV, dtype=torch.bool) if s["mask"] is None else s["mask"].bool()
    loss, coef, filled = 0.0, [], sum(bool(keep[lo:hi].any()) for lo, hi in zip(ends[:-1], ends[1:]))
    for lo, hi in zip(ends[:-1], ends[1:]):
        rows = keep[lo:hi]
        held = max(int(rows.sum()), 1)
        fraction = torch.bincount(s["ids"][lo:hi][rows].reshape(-1).long(), minlength=e).double() / (held * k)
        mean = share[lo:hi][rows].sum(0) / held
        loss = loss + e * (fraction * mean).sum() / max(filled, 1)
        coef.append(case["alpha"] * e * fraction / held / max(filled, 1))
    loss = case["alpha"] * loss
    if op == "balance":
        return loss.detach().reshape(1), None, torch.stack(coef)
    w = score.gather(1, s["ids"].long())
    w = w / w.sum(1, keepdim=True) if case["renorm"] else w
    total = (w * case["scale"] * s["gw"].double()).sum() + loss * s["gl"].double()[0]
    return torch.autograd.grad(total, x)[0]
