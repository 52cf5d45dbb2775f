"""The measured cases of the norm and the 16-bit expert products: their inputs, plain forms, calls and exact values.

The operators on either side of the MoE layer's 16-bit rows, each in a plain torch form (own = False) and as the
library's call (own = True):

  norm             the root-mean-square norm of x + residual: the normed rows, the sum (the next residual), the rows'
                   reciprocal root mean squares and, for a quantised layer, the normed rows' MXFP8 codes and scales;
  norm gradient    the gradient by x (and the residual, which has the same) and by the norm's weight;
  product          out[r] = x[r] w_g^T of the rows r of each expert group, 16-bit operands;
  input gradient   grad_x[r] = grad_out[r] w_g, the same weights contracted over their other dimension;
  weight gradient  grad_w_g = sum over the group's rows r of grad_out[r]^T x[r].
"""

import math

import torch

own = False

DEV = "cuda"
FLOATS = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
NORMS = ("norm", "norm gradient")
EPS = 1e-6
F8MAX = 448.0


# ---- cases ---------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of one request in front of an MXFP8 layer (hidden 7168): the router reads the normed row,
        # the experts its codes
        dict(name="norm 1x7168 mxfp8", op="norm", rows=1, cols=7168, dtype="bf16", residual=True, quant=True),
        # a prefill batch of the prefill workload (8192 tokens)
        dict(name="norm 8192x7168 mxfp8", op="norm", rows=8192, cols=7168, dtype="bf16", residual=True, quant=True),
        # the backward pass of such a batch, with the residual stream's own gradient
        dict(name="norm gradient 8192x7168", op="norm gradient", rows=8192, cols=7168, dtype="bf16", residual=True),
        # a small odd layer: rows and columns that fill no vector, no residual
        dict(name="norm gradient 517x1001", op="norm gradient", rows=517, cols=1001, dtype="fp16", residual=False),
        # the router's logits of one decode step: one row, 256 experts
        dict(name="product 1 row router", op="product", rows=1, groups=1, k=7168, n=256, dtype="bf16", out="fp32",
             skew=0.0),
        # the up projection in decode, a quarter of the decode workload's experts: 128 tokens x topK 8 / 4 = 256 rows
        dict(name="product 256 rows 64 experts", op="product", rows=256, groups=64, k=7168, n=4096, dtype="bf16",
             out="bf16", skew=0.0),
        # a ragged batch: odd row count, an expert without rows, sizes that fill no tile
        dict(name="product 777 rows ragged", op="product", rows=777, groups=5, k=1408, n=2000, dtype="fp16", out="fp16",
             skew=1.0),
        # the up projection of a large batch, 2048 rows an expert
        dict(name="product 32768 rows 16 experts", op="product", rows=32768, groups=16, k=7168, n=4096, dtype="bf16",
             out="bf16", skew=0.0),
        # the gradient by the up projection's input, 256 rows an expert
        dict(name="input gradient 8192 rows", op="input gradient", rows=8192, groups=32, k=7168, n=4096, dtype="bf16",
             out="bf16", skew=0.0),
        # the gradient by the input of a small router with an odd number of experts
        dict(name="input gradient 60 experts", op="input gradient", rows=1000, groups=1, k=2048, n=60, dtype="bf16",
             out="bf16", skew=0.0),
        # the gradient of the down projection's weights of a training batch, 2048 rows an expert
        dict(name="weight gradient 32768 rows", op="weight gradient", rows=32768, groups=16, k=2048, n=7168,
             dtype="bf16", out="bf16", skew=0.0),
        # the gradient of the router's weights: few outputs, many rows, kept in fp32
        dict(name="weight gradient router", op="weight gradient", rows=8192, groups=1, k=7168, n=256, dtype="bf16",
             out="fp32", skew=0.0),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([*NORMS, "product", "input gradient", "weight gradient"])
    top = [work(d) for d in listed() if (d["op"] in NORMS) == (op in NORMS)]
    while True:
        if op in NORMS:
            cols = rng.choice([32 * _between(rng, 1, 512), 32 * _between(rng, 1, 256), _between(rng, 1, 8192)])
            c = dict(op=op, rows=_between(rng, 1, 32768), cols=cols, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     residual=rng.random() < 0.7)
            if op == "norm":
                c["quant"] = cols % 32 == 0 and rng.random() < 0.6
        else:
            step = rng.choice([64, 8, 8, 1])
            c = dict(op=op, rows=_between(rng, 1, 32768), groups=_between(rng, 1, 64),
                     k=step * _between(rng, max(1, 32 // step), 8192 // step),
                     n=step * _between(rng, max(1, 32 // step), 8192 // step), dtype=rng.choice(["bf16", "fp16"]),
                     skew=rng.choice([0.0, 0.0, 0.5, 1.0]))
            c["out"] = rng.choice([c["dtype"], "fp32"])
        w = work(c)
        # a skewed batch's plain form pads every group to the longest
        padded = 0 if op in NORMS else c["rows"] * (1 if c["skew"] == 0 else c["groups"]) * (c["k"] + c["n"])
        if (w["flops"] <= max(t["flops"] for t in top) and w["bytes"] <= max(t["bytes"] for t in top)
                and padded <= 5e8):
            return c


def work(case):
    rows, sz = case["rows"], SIZE[case["dtype"]]
    if case["op"] in NORMS:
        c = case["cols"]
        one = rows * c * sz  # a matrix of rows
        if case["op"] == "norm":  # x, residual in; y, the sum, reciprocals, codes and scales out; weight
            moved = one * (4 if case["residual"] else 2) + rows * 4 + c * sz
            return dict(bytes=moved + (rows * c * 33 / 32 if case["quant"] else 0), flops=rows * c * 6.0)
        # the gradient of y, the sum, reciprocals, the sum's gradient in; both gradients out
        return dict(bytes=one * (4 if case["residual"] else 3) + rows * 4 + c * (sz + 4), flops=rows * c * 9.0)
    g, k, n = min(case["groups"], rows), case["k"], case["n"]
    out = SIZE[case["out"]]
    flops = 2.0 * rows * n * k
    if case["op"] == "product":
        return dict(bytes=(rows * k + g * n * k) * sz + rows * n * out, flops=flops)
    if case["op"] == "input gradient":
        return dict(bytes=(rows * n + g * n * k) * sz + rows * k * out, flops=flops)
    return dict(bytes=rows * (n + k) * sz + case["groups"] * n * k * out, flops=flops)


# ---- inputs --------------------------------------------------------------------------------------------------------
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
    dt = FLOATS[case["dtype"]]
    rows = case["rows"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std).to(dt)

    s = dict(case=case)
    if case["op"] in NORMS:
        cols = case["cols"]
        # a residual stream's rows differ in size, and a few of its channels are much larger than the others
        big = torch.ones((cols,), device=DEV)
        big[torch.randperm(cols, generator=host)[:max(1, cols // 500)].to(DEV)] = 20.0
        stream = torch.randn((rows, cols), generator=gen, device=DEV) * big
        stream = (stream * torch.exp(torch.randn((rows, 1), generator=gen, device=DEV))).to(dt)
        s["w"] = (1.0 + 0.2 * torch.randn((cols,), generator=gen, device=DEV)).to(dt)
        if case["op"] == "norm":
            s["x"] = normal(rows, cols) if case["residual"] else stream
            s["residual"] = stream if case["residual"] else None
            return s
        s["h"] = stream
        s["rstd"] = _rstd(stream.float())
        s["gy"] = normal(rows, cols, std=0.02)
        s["gh"] = normal(rows, cols, std=0.02) if case["residual"] else None
        return s
    groups, k, n = case["groups"], case["k"], case["n"]
    if case["op"] != "weight gradient":
        s["w"] = torch.empty((groups, n, k), dtype=dt, device=DEV)
        for g in range(0, groups, 4):  # a few experts' float weights at a time
            s["w"][g:g + 4] = normal(min(4, groups - g), n, k, std=1.0 / math.sqrt(k))
    if case["op"] != "input gradient":
        s["x"] = normal(rows, k)
    if case["op"] != "product":
        s["g"] = normal(rows, n, std=0.02)
    size = _sizes(case, host) if groups > 1 else torch.tensor([rows])
    end = torch.cumsum(size, 0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), end])
    s["offsets"] = offsets.to(torch.int32).to(DEV) if groups > 1 else None
    s["ends"] = offsets.tolist()
    # the plain form's padding: row of each slot of [groups, longest], whether it is one, slot of each row
    longest = int(size.max())
    slot = (end - size)[:, None] + torch.arange(longest)
    group = torch.repeat_interleave(torch.arange(groups), size)
    s["slot"] = slot.clamp(max=rows - 1).to(DEV)
    s["filled"] = (torch.arange(longest) < size[:, None])[..., None].to(DEV)
    s["place"] = (group * longest + torch.arange(rows) - (end - size)[group]).to(DEV)
    return s


# ---- plain forms ---------------------------------------------------------------------------------------------------
def _rstd(v):
    return 1.0 / torch.sqrt((v * v).mean(1) + EPS)


def _mx(y):
    """MXFP8 (E4M3) codes [R, C] and E8M0 scales [R, C/32 made even, the pad 0] of y (fp32), both as the values that
    they stand for: shared exponent floor(log2 amax) - 8, elements to the nearest, magnitudes above 448 held there."""
    v = y.reshape(y.shape[0], -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    b = (torch.frexp(amax).exponent + 118).clamp(0, 254)  # frexp: amax = m 2^e, m in [0.5, 1)
    b = torch.where(amax > 0, b, 0)
    codes = torch.ldexp(v, 127 - b).clamp(-F8MAX, F8MAX).to(torch.float8_e4m3fn).reshape(y.shape)
    scales = torch.nn.functional.pad(b[:, :, 0].to(torch.uint8), (0, b.shape[1] % 2))
    return codes, scales.view(torch.float8_e8m0fnu)


def _norm(s):
    x, dt = s["x"], s["x"].dtype
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(dt)
    v = h.float()
    rstd = _rstd(v)
    y = (v * rstd[:, None] * s["w"].float()).to(dt)
    return (y, h, rstd, *_mx(y.float())) if s["case"]["quant"] else (y, h, rstd)


def _norm_gradient(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    gy = s["gy"].float()
    gw = gy * s["w"].float()
    gx = s["rstd"][:, None] * (gw - xhat * (gw * xhat).mean(1, keepdim=True))
    if s["gh"] is not None:
        gx = gx + s["gh"].float()
    return gx.to(s["h"].dtype), (gy * xhat).sum(0)


def _padded(t, s):
    return t.float()[s["slot"]]


def _product(s, rows, w):
    out = torch.bmm(_padded(rows, s), w)
    return out.reshape(-1, w.shape[2])[s["place"]].to(FLOATS[s["case"]["out"]])


def _weight_gradient(s):
    g = torch.where(s["filled"], _padded(s["g"], s), 0.0)
    return torch.bmm(g.transpose(1, 2), _padded(s["x"], s)).to(FLOATS[s["case"]["out"]])


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "norm":
            return _norm(s)
        if op == "norm gradient":
            return _norm_gradient(s)
        if op == "product":
            return _product(s, s["x"], s["w"].float().transpose(1, 2))
        if op == "input gradient":
            return _product(s, s["g"], s["w"].float())
        return _weight_gradient(s)
    import routing_permute_mxfp8_amd as rp
    if op == "norm":
        y, h, rstd, codes, scales = rp.rms_norm(s["x"], s["w"], s["residual"], eps=EPS,
                                                quant_mode=rp.QUANT_E4M3 if case["quant"] else rp.QUANT_NONE)
        if case["quant"]:  # the values that the bytes stand for
            return y, h, rstd, codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
        return y, h, rstd
    if op == "norm gradient":
        return rp.rms_norm_backward(s["gy"], s["h"], s["w"], s["rstd"], grad_h=s["gh"])
    out = FLOATS[case["out"]]
    if op == "product":
        return rp.grouped_matmul(s["x"], s["w"], s["offsets"], out_dtype=out)
    if op == "input gradient":
        return rp.grouped_matmul(s["g"], s["w"], s["offsets"], transpose_w=True, out_dtype=out)
    return rp.grouped_matmul_wgrad(s["g"], s["x"], s["offsets"], out_dtype=out).reshape(case["groups"], case["n"], case["k"])


# ---- from the definitions, in 64 bits ------------------------------------------------------------------------------
def _nearest_mx(y):
    """y (64 bits) as MXFP8 element values and scales: steps of 2^-3 of each value's own power of two (2^-9 at least)
    over the power of two that brings its 32-group's largest magnitude into [256, 512)."""
    g = y.reshape(-1, 32)
    top = g.abs().max(1, keepdim=True).values
    scale = torch.exp2((torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 8).clamp(min=-127))
    scale = torch.where(top > 0, scale, 2.0 ** -127)
    v = g / scale
    step = torch.exp2(torch.floor(torch.log2(torch.where(v != 0, v.abs(), 1.0))).clamp(min=-6) - 3)
    v = (torch.round(v / step) * step).clamp(-F8MAX, F8MAX)
    scales = scale.reshape(y.shape[0], -1)
    pad = scales.new_full((y.shape[0], scales.shape[1] % 2), 2.0 ** -127)
    return v.reshape(y.shape), torch.cat([scales, pad], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        dt = s["x"].dtype
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(dt).double()  # the sum is kept, and normed, in the stream's type
        rms = torch.linalg.vector_norm(h, dim=1).square() / case["cols"] + EPS
        y = s["w"].double() * h / rms.sqrt()[:, None]
        if not case["quant"]:
            return y, h, rms ** -0.5
        return y, h, rms ** -0.5, *_nearest_mx(y.to(dt).double())  # the codes are those of the rows as they are kept
    if op == "norm gradient":
        h, w = s["h"].double().requires_grad_(True), s["w"].double().requires_grad_(True)
        y = torch.nn.functional.normalize(h, dim=1) * math.sqrt(case["cols"])  # eps as a factor below
        mean = (h * h).sum(1, keepdim=True) / case["cols"]
        y = y * torch.sqrt(mean / (mean + EPS)) * w
        loss = (y * s["gy"].double()).sum()
        if s["gh"] is not None:
            loss = loss + (h * s["gh"].double()).sum()
        return torch.autograd.grad(loss, (h, w))
    ends = list(zip(s["ends"][:-1], s["ends"][1:]))
    if op == "weight gradient":
        out = torch.zeros((case["groups"], case["n"], case["k"]), dtype=torch.float64, device=DEV)
        for g, (lo, hi) in enumerate(ends):
            out[g] = s["g"][lo:hi].double().T @ s["x"][lo:hi].double()
        return out
    left, width = (s["x"], case["n"]) if op == "product" else (s["g"], case["k"])
    out = torch.zeros((case["rows"], width), dtype=torch.float64, device=DEV)
    for g, (lo, hi) in enumerate(ends):
        w = s["w"][g].double()
        out[lo:hi] = left[lo:hi].double() @ (w.T if op == "product" else w)
    return out
