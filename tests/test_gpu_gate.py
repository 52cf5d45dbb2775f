"""The router on the GPU (gate_topk, balance_loss, gate_backward) against the float64 oracle.

Chosen ids and counts have to be equal. Bounds on values, u = 2^-24 being fp32's rounding:
* a score exp(l - m) / sum: the argument is off by |l - m| 2 u (subtraction, multiplication by
  log2 e), V_EXP_F32 and the reciprocal by 2 u each, the sum of up to 1024 terms by 22 u
  (16 in a lane, 6 steps over the wave): for |l - m| <= 30 under (60 + 26) u + 2^-40 < 2^-17
  relative; a sigmoid's 1 / (1 + exp(-l)) less. A weight is one or a quotient of two such
  scores: WEIGHT = 2^-15 relative.
* gradients: sums of at most 1024 products of such scores, 2^-17 and 32 u each:
  GRAD = 2^-14 of the sum of the terms' magnitudes, and the rounding to the logits' type.
* the loss: positive terms, 2^-17 each, sums over a few rows in fp32: 2^-15 relative."""
import numpy as np
import pytest
import torch

import routing_permute_mxfp8_amd as rp
from gpu_support import DEV, say
from oracle import gate

pytestmark = pytest.mark.gpu

SCORING = {"softmax": rp.GATE_SOFTMAX, "sigmoid": rp.GATE_SIGMOID}
WEIGHT, GRAD, LOSS = 2.0 ** -15, 2.0 ** -14, 2.0 ** -15
TYPES = [torch.float32, torch.float16, torch.bfloat16]


def logits_of(n, e, dtype, seed=0, spread=2.0, dead=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, e)) * spread
    if dead:
        x[rng.random((n, e)) < dead] = -np.inf
        x[rng.random((n, e)) < dead / 4] = np.nan
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def check_gate(x, k, scoring, bias=None, groups=1, topk_groups=1, renorm=True, scale=1.0):
    say(f"gate_topk {tuple(x.shape)} {x.dtype} k={k} {scoring} bias={bias is not None} groups={groups}/{topk_groups}")
    ids, w = rp.gate_topk(x.to(DEV), k, scoring=SCORING[scoring], bias=None if bias is None else bias.to(DEV),
                          num_groups=groups, topk_groups=topk_groups, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    want_ids, want = gate.topk(x.double().numpy(), k, scoring, None if bias is None else bias.double().numpy(), groups,
                               topk_groups, renorm, scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = w.cpu().double().numpy()
    # fp32's range ends at 2^-126 (a score below is flushed or denormal: its quotients are not bounded)
    assert np.all(np.abs(got - want) <= WEIGHT * np.abs(want) + 2.0 ** -100 * scale)
    return ids, w


@pytest.mark.parametrize("e,k", [(1, 1), (2, 1), (7, 3), (60, 4), (64, 8), (65, 8), (100, 10), (128, 6), (255, 8),
                                 (256, 8), (257, 9), (384, 32), (512, 8), (1000, 16), (1024, 32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gate_sizes(e, k, scoring):
    for i, (n, dtype) in enumerate([(1, torch.float32), (5, torch.bfloat16), (37, torch.float16)]):
        x = logits_of(n, e, dtype, seed=e + i)
        check_gate(x, k, scoring, renorm=i != 1, scale=(1.0, 2.5, 0.5)[i])
        check_gate(x, k, scoring, bias=torch.randn(e, generator=torch.Generator().manual_seed(e)) * 0.1)


@pytest.mark.parametrize("e,k,groups,topk_groups", [(256, 8, 8, 4), (256, 8, 8, 8), (60, 4, 12, 2), (64, 1, 64, 1),
                                                    (64, 5, 64, 5), (6, 3, 2, 1), (160, 6, 8, 3), (1024, 8, 32, 7),
                                                    (1023, 20, 3, 1), (48, 16, 3, 1), (100, 4, 50, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_gate_groups(e, k, groups, topk_groups, scoring, biased):
    for n, dtype, dead in [(33, torch.float32, 0.0), (20, torch.bfloat16, 0.0), (16, torch.float32, 0.4)]:
        x = logits_of(n, e, dtype, seed=7 * e + groups, dead=dead)
        bias = torch.randn(e, generator=torch.Generator().manual_seed(groups)) * 0.1 if biased else None
        check_gate(x, k, scoring, bias, groups, topk_groups)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gate_ranks_next_to_each_other(scoring):
    """Biases that bring every rank of a row within a rounding of one value: 32-bit ranks
    cannot order them, the exact ones can. Every expert's bias cancels one row's scores."""
    for e, k, groups, keep in [(64, 8, 1, 1), (256, 8, 8, 4), (300, 12, 10, 2)]:
        for seed in range(4):
            x = logits_of(1, e, torch.float32, seed=seed)
            s = gate.scores(x.double().numpy(), scoring)[0]
            bias = torch.from_numpy((0.5 - s).astype(np.float32))
            check_gate(x.repeat(3, 1), k, scoring, bias, groups, keep)


def test_gate_ties_and_infinities():
    """Equal logits go to the lowest index; -inf, NaN and rows of them are chosen last with
    weight 0; +inf and the types' lowest values stay finite."""
    e = 130
    for dtype in TYPES:
        rng = np.random.default_rng(3)
        x = torch.from_numpy(rng.integers(-2, 3, (24, e)).astype(np.float32))
        x[3] = -np.inf
        x[4] = np.nan
        x[5, 10:] = -np.inf
        x[6] = 0.0
        x = x.to(dtype)
        x[7] = torch.finfo(dtype).min
        x[8, ::3] = torch.finfo(dtype).min
        x[9, 77] = torch.finfo(dtype).max
        for scoring in ("softmax", "sigmoid"):
            for renorm in (True, False):
                check_gate(x, 12, scoring, renorm=renorm)
            check_gate(x, 12, scoring, bias=torch.zeros(e))
            check_gate(x, 12, scoring, groups=10, topk_groups=2)
        x[10, 5] = np.inf
        ids, w = rp.gate_topk(x.to(DEV), 3)
        assert int(ids[10, 0]) == 5 and float(w[10, 0]) == 1.0 and bool(torch.isfinite(w).all())


def test_gate_misaligned_rows_and_out_of_order_streams():
    base = logits_of(1, 41 * 64 + 1, torch.float32, seed=2).reshape(-1).to(DEV)
    x = base[1:].reshape(41, 64)      # rows of 64 floats, 4 bytes off a 16-byte line
    ids, w = rp.gate_topk(x, 6)
    want_ids, want_w = rp.gate_topk(x.clone(), 6)
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
    x = logits_of(1, 41 * 256 + 1, torch.bfloat16, seed=2).reshape(-1).to(DEV)[1:].reshape(41, 256)
    assert torch.equal(rp.gate_topk(x, 6)[0], rp.gate_topk(x.clone(), 6)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = rp.gate_topk(x, 6)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other[0], rp.gate_topk(x, 6)[0])


def test_gate_no_rows():
    x = torch.empty((0, 32), device=DEV)
    ids, w = rp.gate_topk(x, 4)
    assert tuple(ids.shape) == (0, 4) and tuple(w.shape) == (0, 4)
    loss, counts, coef = rp.balance_loss(x, ids, seq_offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert float(loss) == 0.0 and int(counts.abs().sum()) == 0 and float(coef.abs().sum()) == 0.0
    assert tuple(rp.gate_backward(x, ids, w).shape) == (0, 32)


def seqs_of(n, kind):
    """(offsets, mask) of a ragged or padded batch of n rows."""
    rng = np.random.default_rng(n)
    if kind == "one":
        return None, None
    if kind == "mask":
        return None, (rng.random(n) < 0.7).astype(np.uint8)
    if kind == "nothing counts":
        return None, np.zeros(n, dtype=np.uint8)
    if kind == "ragged":   # empty sequences at both ends and inside, rows behind the last one
        end = max(n - 3, 0)
        cut = np.sort(rng.integers(0, end + 1, 3))
        return np.array([0, 0, *cut, cut[-1], end, end], dtype=np.int32), None
    # many short sequences, some of them masked whole
    off = np.minimum(np.arange(0, n + 3, 3), n).astype(np.int32)
    return off, (rng.random(n) < 0.3).astype(np.uint8)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_balance(x, k, scoring, kind, alpha=0.01):
    n, e = x.shape
    off, mask = seqs_of(n, kind)
    ids = gate.topk(x.double().numpy(), k, scoring)[0]
    say(f"balance_loss {n}x{e} {x.dtype} k={k} {scoring} {kind}")
    loss, counts, coef = rp.balance_loss(x.to(DEV), dev(ids), scoring=SCORING[scoring], seq_offsets=dev(off),
                                         row_mask=dev(mask), alpha=alpha)
    torch.cuda.synchronize()
    wl, wc, wf = gate.balance(x.double().numpy(), ids, scoring, off, mask, alpha)
    assert np.array_equal(counts.cpu().numpy(), wc)
    assert np.all(np.abs(coef.cpu().double().numpy() - wf) <= (2 + 2.0 ** -10) * 2.0 ** -24 * wf)   # alpha and the result rounded
    assert abs(float(loss) - wl) <= LOSS * wl
    again = rp.balance_loss(x.to(DEV), dev(ids), scoring=SCORING[scoring], seq_offsets=dev(off), row_mask=dev(mask),
                            alpha=alpha)
    assert torch.equal(again[0], loss)   # sums in a fixed order
    return ids, off, mask, coef


@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (1, 256, 8), (3, 7, 2), (64, 60, 4), (517, 256, 8), (1000, 100, 5),
                                   (40, 1024, 32), (5000, 64, 6)])
@pytest.mark.parametrize("kind", ["one", "mask", "nothing counts", "ragged", "short"])
def test_balance(n, e, k, kind):
    for i, scoring in enumerate(("softmax", "sigmoid")):
        check_balance(logits_of(n, e, TYPES[(n + i) % 3], seed=n), k, scoring, kind)


def check_backward(x, k, scoring, kind, renorm, parts):
    n, e = x.shape
    ids, off, mask, coef = check_balance(x, k, scoring, kind, alpha=0.5)
    rng = np.random.default_rng(n + e)
    gw = rng.standard_normal((n, k)).astype(np.float32) if "w" in parts else None
    gl = np.array([1.7], dtype=np.float32) if "l" in parts else None
    say(f"gate_backward {n}x{e} {x.dtype} k={k} {scoring} {kind} renorm={renorm} {parts}")
    got = rp.gate_backward(x.to(DEV), dev(ids), dev(gw), scoring=SCORING[scoring], renormalize=renorm, scale=2.0,
                           grad_loss=dev(gl), coef=coef if gl is not None else None, seq_offsets=dev(off),
                           row_mask=dev(mask))
    torch.cuda.synchronize()
    want, mag = gate.backward(x.double().numpy(), ids, scoring, gw, renorm, 2.0, gl,
                              coef.cpu().double().numpy(), off, mask)
    assert got.dtype == x.dtype
    half = torch.finfo(x.dtype).eps / 2
    # (fp16's subnormal step is 2^-24)
    bound = GRAD * mag + half * (np.abs(want) + GRAD * mag) + (2.0 ** -24 if x.dtype == torch.float16 else 2.0 ** -120)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= bound)


@pytest.mark.parametrize("n,e,k", [(1, 1, 1), (1, 256, 8), (5, 7, 2), (61, 60, 4), (130, 256, 8), (300, 100, 5),
                                   (17, 1024, 32), (9, 300, 9)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["one", "mask", "ragged", "short"])
def test_backward(n, e, k, scoring, kind):
    for i, parts in enumerate(("w", "l", "wl")):
        x = logits_of(n, e, TYPES[(n + i) % 3], seed=n + i)
        check_backward(x, k, scoring, kind, renorm=(n + i) % 2 == 0, parts=parts)


def test_backward_of_rows_without_experts():
    """Experts taken out get gradient 0, and a row of them is all zeros."""
    x = logits_of(40, 70, torch.float32, seed=5, dead=0.3)
    x[7] = -np.inf
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_backward(x, 6, scoring, "ragged", renorm, "wl")
    ids = gate.topk(x.double().numpy(), 6, "softmax")[0]
    got = rp.gate_backward(x.to(DEV), dev(ids), torch.ones((40, 6), device=DEV))
    assert bool((got[7] == 0).all()) and bool((got[x.to(DEV) == -np.inf] == 0).all())
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_backward_against_differences(scoring):
    """The GPU gradient against central differences of the GPU's own forward calls: the fp32
    weights and loss are off by 2^-17 of their size, so with a step of 2^-5 the quotient is off
    by 2^-17 sum |gw w| / 2^-5 and its truncation by h^2 / 6 sum |f'''|, under 2^-12 of the same sum each."""
    n, e, k, h = 1, 12, 4, 2.0 ** -5
    x = logits_of(n, e, torch.float32, seed=11)
    ids = dev(gate.topk(x.double().numpy(), k, scoring)[0])
    gw = torch.randn((n, k), generator=torch.Generator().manual_seed(1))

    def total(y):   # the weights of the chosen experts (their choice held fixed) and the loss
        w_all, i_all = rp.gate_topk(y, e, scoring=SCORING[scoring], renormalize=False)[::-1]
        s = torch.zeros((n, e), device=DEV).scatter_(1, i_all.long(), w_all)
        w = s.gather(1, ids.long())
        w = (w / w.sum(1, keepdim=True)).cpu().double()
        return float((w * gw.double()).sum()) + float(rp.balance_loss(y, ids, scoring=SCORING[scoring])[0])

    coef = rp.balance_loss(x.to(DEV), ids, scoring=SCORING[scoring])[2]
    got = rp.gate_backward(x.to(DEV), ids, gw.to(DEV), scoring=SCORING[scoring], coef=coef,
                           grad_loss=torch.ones(1, device=DEV)).cpu()
    size = float(gw.abs().max()) + float(coef.max())
    for i in range(e):
        y, z = x.clone(), x.clone()
        y[0, i] += h
        z[0, i] -= h
        diff = (total(y.to(DEV)) - total(z.to(DEV))) / (2 * h)
        assert abs(diff - float(got[0, i])) <= 2.0 ** -10 * size


def test_gate_step_captured_and_replayed():
    """Choice, loss and gradient in one captured graph, replayed on changed logits with eager
    work between the replays; two graphs live at once and keep their own workspaces."""
    n, e, k = 700, 64, 6
    off = torch.tensor([0, 100, 350, 700], dtype=torch.int32, device=DEV)
    gl = torch.ones(1, device=DEV)

    def step(x, gw):
        ids, w = rp.gate_topk(x, k)
        loss, counts, coef = rp.balance_loss(x, ids, seq_offsets=off, alpha=0.1)
        return ids, w, loss, counts, coef, rp.gate_backward(x, ids, gw, grad_loss=gl, coef=coef, seq_offsets=off)

    held = []
    for g in range(2):
        x = logits_of(n, e, torch.float32, seed=g).to(DEV)
        gw = torch.randn((n, k), device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x, gw)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x, gw)
        held.append((graph, x, gw, out))
    for r in range(4):
        for g, (graph, x, gw, out) in enumerate(held):
            x.copy_(logits_of(n, e, torch.float32, seed=10 * r + g))
            graph.replay()
        torch.cuda.synchronize()
        for graph, x, gw, out in held:
            for a, b in zip(out, step(x, gw)):
                assert torch.equal(a, b)


def test_gate_feeds_the_routing():
    """The router's ids go through init_routing as they are, and their counts are its counts."""
    n, e, k, h = 300, 24, 3, 256
    x = torch.randn((n, h), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).to(DEV)
    logits = logits_of(n, e, torch.bfloat16, seed=4).to(DEV)
    ids, w = rp.gate_topk(logits, k, scoring=rp.GATE_SIGMOID, num_groups=4, topk_groups=2)
    _, counts, _ = rp.balance_loss(logits, ids, scoring=rp.GATE_SIGMOID)
    tokens = rp.init_routing(x, ids, e, quant_mode=rp.QUANT_MXFP4)[2]
    assert torch.equal(tokens, counts[0].long())


@pytest.mark.parametrize("n,e,seqs", [(30000, 256, 1), (30000, 100, 2), (20000, 40, 1), (9000, 700, 1)])
def test_balance_of_many_partials(n, e, seqs):
    """Long sequences: hundreds of partial sums each, joined on few and on many blocks."""
    k = 6
    rng = np.random.default_rng(n + e)
    x = torch.from_numpy(rng.standard_normal((n, e)).astype(np.float32))
    ids = torch.from_numpy(np.argsort(rng.random((n, e)), axis=1)[:, :k].astype(np.int32))
    off = None if seqs == 1 else [0, 3, n]
    mask = rng.random(n) > 0.1
    say(f"balance_loss {n}x{e} seqs={seqs}")
    loss, counts, coef = rp.balance_loss(x.to(DEV), ids.to(DEV), alpha=0.5, row_mask=torch.from_numpy(mask).to(DEV),
                                         seq_offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV))
    p = torch.softmax(x.double(), dim=1).numpy()
    bounds = off or [0, n]
    total, filled = 0.0, sum(bool(mask[lo:hi].any()) for lo, hi in zip(bounds[:-1], bounds[1:]))
    for b, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        m = mask[lo:hi]
        rows = int(m.sum())
        c = np.bincount(ids.numpy()[lo:hi][m].reshape(-1), minlength=e)
        f = 0.5 * e * c / (k * rows * rows * filled)
        assert np.array_equal(counts[b].cpu().numpy(), c)
        # one rounding to fp32 of a float64 product of a few factors
        assert np.all(np.abs(coef[b].cpu().double().numpy() - f) <= 2.0 ** -23 * f)
        total += float((f * p[lo:hi][m].sum(axis=0)).sum())
    # a score is off by at most (|l - m| + 12) 2^-23 of itself, |l - m| < 12; a wave's fp32 sums of
    # at most 64 rows by 64 2^-24; then the rounding of the loss
    assert abs(float(loss) - total) <= (24 * 2.0 ** -23 + 64 * 2.0 ** -24 + 2.0 ** -24) * total


BIASES = {
    "one NaN": lambda e: {e // 3: np.nan},
    "NaN": lambda e: {i: np.nan for i in range(0, e, 3)},
    "all NaN": lambda e: {i: np.nan for i in range(e)},
    "-inf": lambda e: {i: -np.inf for i in range(1, e, 2)},
    "+inf": lambda e: {1: np.inf, e - 1: np.inf},
    "all of them": lambda e: {0: np.nan, 1: -np.inf, 2: np.inf, e // 2: np.inf, e - 2: np.nan, e - 1: -np.inf},
    "largest": lambda e: {i: float(np.finfo(np.float32).max) * (-1) ** i for i in range(0, e, 5)},
}


@pytest.mark.parametrize("e,k,groups,topk_groups", [(7, 5, 1, 1), (60, 8, 1, 1), (128, 8, 4, 2), (256, 8, 1, 1),
                                                    (256, 8, 8, 4), (60, 9, 1, 1), (160, 6, 8, 3), (300, 12, 1, 1)])
@pytest.mark.parametrize("kind", list(BIASES))
def test_gate_bias_without_a_value(e, k, groups, topk_groups, kind):
    """NaN in the bias is -inf: such experts come last, in index order, whether 16 lanes or the
    whole wave choose; the ids stay distinct and every place is written."""
    bias = torch.randn(e, generator=torch.Generator().manual_seed(e)) * 0.1
    for i, v in BIASES[kind](e).items():
        bias[i] = v
    for scoring in ("softmax", "sigmoid"):
        for dtype, dead in [(torch.float32, 0.0), (torch.bfloat16, 0.3)]:
            x = logits_of(9, e, dtype, seed=e + k, dead=dead)
            ids, w = check_gate(x, k, scoring, bias, groups, topk_groups)
            assert all(len(set(row)) == k for row in ids.tolist()) and bool(torch.isfinite(w).all())


@pytest.mark.parametrize("e", [256, 512])
@pytest.mark.parametrize("equal", [True, False])
def test_balance_of_one_long_sequence_among_many(e, equal):
    """1023 sequences of three rows and one of 32768, where a block may get a whole sequence:
    what its lanes add in fp32 must not grow with the sequence. The loss of rows that all chose
    one expert is a single expert's sum. With equal rows every addition rounds the same way:
    2048 of them (8192 above 256 experts) are off by up to 2^-15 (2^-13).
    Bound: a score by 2^-17.5 (|l - m| < 12: (24 + 22 + 8) 2^-24; the same for equal rows), at
    most 64 rows added in fp32 by 2^-18, roundings of the partial sum and of the loss 2^-23."""
    rng = np.random.default_rng(e)
    long, short = 32768, 1023
    n = long + 3 * short
    rows = rng.standard_normal((n, e)).astype(np.float32) * 1.5
    if equal:
        rows[:] = rows[0]
    off = np.array([0, *(3 * np.arange(1, 513)), 3 * 512 + long,
                    *(3 * 512 + long + 3 * np.arange(1, 512))], dtype=np.int32)
    assert off[-1] == n and off.size == 1025
    mask = np.zeros(n, dtype=np.uint8)
    mask[3 * 512:3 * 512 + long] = 1   # only the long one counts
    p = torch.softmax(torch.from_numpy(rows[3 * 512:3 * 512 + long]).double(), 1).mean(0).numpy()
    x = torch.from_numpy(rows).to(DEV)
    for expert in (0, 7, e // 3, e // 2 + 1, e - 60, e - 37, e - 2, e - 1):
        say(f"balance_loss long sequence e={e} equal={equal} expert={expert}")
        ids = torch.full((n, 1), expert, dtype=torch.int32, device=DEV)
        loss, counts, _ = rp.balance_loss(x, ids, seq_offsets=dev(off), row_mask=dev(mask))
        assert int(counts[512, expert]) == long and int(counts.sum()) == long
        want = e * float(p[expert])
        assert abs(float(loss) - want) <= (2.0 ** -17.5 + 2.0 ** -18 + 2.0 ** -23) * want


def repeated(base, rows):
    """`rows` rows: those of base over and over."""
    x = base.repeat(-(-rows // base.shape[0]), 1)
    return x[:rows]


def assert_repeats(got, want):
    """got's rows are want's rows over and over."""
    n = want.shape[0]
    whole = got.shape[0] // n * n
    assert bool((got[:whole].view(-1, *want.shape) == want).all()) and torch.equal(got[whole:], want[:got.shape[0] - whole])


def test_gate_of_more_rows_than_a_launch_takes():
    """2^26 rows at 64 lanes each and 2^28 at 16 are more threads than one launch has."""
    n, e, k = (1 << 26) + 5, 10, 9
    base = logits_of(1 << 12, e, torch.bfloat16, seed=1).to(DEV)
    say(f"gate_topk {n}x{e} k={k}")
    ids, w = rp.gate_topk(repeated(base, n), k)
    want = rp.gate_topk(base, k)
    assert_repeats(ids, want[0])
    assert_repeats(w, want[1])
    del ids, w
    n, e, k = (1 << 28) + 7, 2, 1
    base = logits_of(1 << 12, e, torch.bfloat16, seed=2).to(DEV)
    x = repeated(base, n)
    say(f"gate_topk {n}x{e} k={k}")
    ids, w = rp.gate_topk(x, k, renormalize=False)
    want = rp.gate_topk(base, k, renormalize=False)
    assert_repeats(ids, want[0])
    assert_repeats(w, want[1])


def test_backward_of_more_rows_than_a_launch_takes():
    """The same for the gradient, with sequences that begin and end behind the first launch's rows
    and a mask."""
    n, e, k = (1 << 28) + 7, 2, 1
    base = logits_of(1 << 12, e, torch.bfloat16, seed=2).to(DEV)
    x = repeated(base, n)
    ids = rp.gate_topk(base, k)[0]
    gl = torch.ones(1, device=DEV)
    cut = [0, 1 << 27, (1 << 28) - 4096, 1 << 28]   # multiples of the period; the last 7 rows belong to none
    off = torch.tensor(cut, dtype=torch.int32, device=DEV)
    coef = torch.tensor([[0.25, 0.5], [1.0, -1.0], [2.0, 0.125]], device=DEV)
    mask = (torch.arange(1 << 12, device=DEV) % 5 != 0).to(torch.uint8)
    gw = torch.randn((1 << 12, k), generator=torch.Generator().manual_seed(0)).to(DEV)
    say(f"gate_backward {n}x{e} k={k}")
    got = rp.gate_backward(x, repeated(ids, n), repeated(gw, n), renormalize=False, grad_loss=gl, coef=coef,
                           seq_offsets=off, row_mask=repeated(mask[:, None], n)[:, 0].contiguous())
    del x
    for b in range(3):
        want = rp.gate_backward(base, ids, gw, renormalize=False, grad_loss=gl, coef=coef[b:b + 1], row_mask=mask)
        assert_repeats(got[cut[b]:cut[b + 1]], want)
    assert torch.equal(got[1 << 28:], rp.gate_backward(base, ids, gw, renormalize=False)[:7])


@pytest.mark.parametrize("e,k", [(60, 4), (256, 8), (300, 4)])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_where_the_scores_are_tiny(e, k, renorm):
    """Sigmoid scores near fp32's smallest (2^-126 = exp(-87.3)) under large gradients: the
    quotients by their sums are of ordinary size, the reciprocals of these sums are not.
    A score's exponent is off by 87 log2 e (2^-24 + 2^-25) and so the score by under 2^-16.8, a
    quotient of two by 2^-15.8, the differences of at most k + 1 such terms by no more of the sum of
    their magnitudes: within GRAD. A score below 2^-126 is 0 in fp32 (here exp(-120) = 2^-173): every
    term of its own element has it as a factor, so that element may be off by all of its magnitude
    (some 2^-46 of the others'); in the row's sums, over 2^-126 each, it is missing by under 2^-40."""
    n = 33
    rng = np.random.default_rng(e)
    x = torch.from_numpy(rng.uniform(-87.2, -84.0, (n, e)).astype(np.float32))
    x[1] = -87.25
    x[2, ::2] = -120.0   # scores of 0
    ids = gate.topk(x.double().numpy(), k, "sigmoid")[0]
    gw = (rng.standard_normal((n, k)) * 1000).astype(np.float32)
    coef = torch.from_numpy(rng.random((1, e)).astype(np.float32) * 1000)
    for parts in ("w", "l", "wl"):
        say(f"gate_backward tiny scores e={e} k={k} renorm={renorm} {parts}")
        gl = np.array([3.0], dtype=np.float32) if "l" in parts else None
        got = rp.gate_backward(x.to(DEV), dev(ids), dev(gw) if "w" in parts else None, scoring=rp.GATE_SIGMOID,
                               renormalize=renorm, grad_loss=dev(gl), coef=coef.to(DEV) if gl is not None else None)
        want, mag = gate.backward(x.double().numpy(), ids, "sigmoid", gw if "w" in parts else None, renorm, 1.0, gl,
                                  coef.double().numpy())
        got = got.cpu().double().numpy()
        assert np.all(np.isfinite(got))
        own = np.where(gate.scores(x.double().numpy(), "sigmoid") < 2.0 ** -126, 1.0, GRAD)
        assert np.all(np.abs(got - want) <= own * mag + 2.0 ** -24 * (np.abs(want) + GRAD * mag) + 2.0 ** -120)


@pytest.mark.parametrize("e,k", [(8, 4), (60, 8), (256, 32), (300, 6)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_of_an_expert_chosen_twice(e, k, scoring, renorm):
    """An id that stands in several places of a row gets the sum of their gradients."""
    n = 21
    rng = np.random.default_rng(e + k)
    x = logits_of(n, e, torch.float32, seed=e)
    ids = rng.integers(0, e, (n, k)).astype(np.int32)
    ids[0] = 3
    ids[1, 1] = ids[1, 0]
    ids[2, -1] = ids[2, 0]
    gw = rng.standard_normal((n, k)).astype(np.float32)
    say(f"gate_backward repeated ids e={e} k={k} {scoring} renorm={renorm}")
    call = lambda: rp.gate_backward(x.to(DEV), dev(ids), dev(gw), scoring=SCORING[scoring], renormalize=renorm)
    got = call()
    want, mag = gate.backward(x.double().numpy(), ids, scoring, gw, renorm)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= GRAD * mag + 2.0 ** -24 * (np.abs(want) + GRAD * mag) + 2.0 ** -120)
    for _ in range(3):
        assert torch.equal(got, call())
