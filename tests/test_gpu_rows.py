"""Row exchanges on the GPU against the oracle in 64 bits.

Error bounds, with u = 2^-24 (float32) and h = eps / 2 of an output's type:
  - route weights are computed in 64 bits and rounded once: u relative.  Only
    the sum of a softmax over all E experts is a float32 one: each exponential
    is off by (1.25 t + 2) u for t below the largest logit, whose mean under
    the softmax is at most about log E < 7, (9 + 2) u in all; each lane adds up
    V <= min(E / 8 + 4, 32) of them and eight or 64 lanes join, V + 6 roundings
    of u: (V + 17) u relative;
  - a sum of n float32 terms in any order is off by at most n u times the sum
    of their absolute values (first order; the factor 1.01 covers the rest);
  - an output in type T adds h of its own value.
Copies, choices, slots and sums in the documented order are compared bit for bit.
"""

import math
import threading

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from gpu_util import session
from oracle import rows as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}  # half a step below the normal range, and more


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g) * std).to(TYPES[dtype])


def dev(ts):
    return [t.to(DEV) for t in ts]


def f64(ts):
    return [t.detach().cpu().double().numpy() for t in ts]


def ints(ts):
    return [t.detach().cpu().numpy() for t in ts]


def near(got, want, bound, what):
    got, want, bound = np.asarray(got, np.float64), np.asarray(want, np.float64), np.asarray(bound, np.float64)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, not {want.shape}"
    if got.size == 0:
        return
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - want) - bound
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, f"{what}: at {i} got {got[i]!r} want {want[i]!r}, bound {bound[i]!r}"


def shifted(ts, off):
    """The same tensors `off` elements into larger ones (rows off the 16-byte grid)."""
    out = []
    for t in ts:
        big = torch.empty(t.numel() + off, dtype=t.dtype, device=t.device)
        big[off:].copy_(t.reshape(-1))
        out.append(big[off:].view(t.shape))
    return out


# ---------------------------------------------------------------- routing

def check_route(logits, top_k, dtype, out=None, **kw):
    R = len(logits)
    l = dev(logits)
    bias = kw.pop("bias", None)
    with session(R):
        w, e = rr.route(l, top_k, bias=None if bias is None else bias.to(DEV), out=out, **kw)
        torch.cuda.synchronize()
    want_w, want_e = orc.route(f64(logits), top_k, bias=None if bias is None else bias.double().numpy(), **kw)
    u = 1.0001 * U
    if kw.get("score", "softmax") == "softmax" and not kw.get("renormalize", True):
        u += (min(logits[0].shape[1] / 8 + 4, 32) + 17) * U
    for r in range(R):
        assert np.array_equal(ints(e)[r], want_e[r]), f"rank {r}: choices differ"
        near(f64(w)[r], want_w[r], u * np.abs(want_w[r]) + 2.0 ** -149, f"weights of rank {r}")
    return w, e


def check_route_grad(logits, experts, dtype, score, renormalize, scale, seed):
    R = len(logits)
    g = gen(seed)
    dw = [normal(g, *e.shape) for e in experts]
    with session(R):
        d = rr.route_grad(dev(logits), dev(experts), dev(dw), score=score, renormalize=renormalize, scale=scale)
        torch.cuda.synchronize()
    x, ex, dwn = f64(logits), ints(experts), f64(dw)
    want = orc.route_grad(x, ex, dwn, score=score, renormalize=renormalize, scale=scale)
    for r in range(R):
        # each chosen expert's part is rounded to float32 before they are added
        part = np.zeros_like(want[r])
        for t in range(x[r].shape[0]):
            s = orc._scores(x[r][t], score)
            ok = [k for k in range(ex[r].shape[1]) if ex[r][t, k] >= 0]
            p = np.array([s[ex[r][t, k]] for k in ok])
            gg = scale * np.array([dwn[r][t, k] for k in ok])
            if not ok:
                continue
            if renormalize:
                q = p / p.sum()
                parts = q * (np.abs(gg) + np.abs((gg * q).sum()))
            else:
                parts = np.abs(gg * p)
                if score == "softmax":
                    # p is the exponential in 64 bits over the float32 sum of all E, which is
                    # off by (V + 17) u as in the weights (above): no more than E / 8 + 4 sums
                    # a lane and three to six over the lanes, of exponentials off by
                    # (t + 2) u; the bound below counts 2 u for each unit
                    parts = parts * (1 + (min(x[r].shape[1] / 8 + 4, 32) + 17) / 2)
            for k, v in zip(ok, parts):
                part[t, ex[r][t, k]] += v
            if score == "softmax" and not renormalize:
                # s in float32: expf of a rounded difference, over a float32 sum of E of them
                E = x[r].shape[1]
                rel = 2 + np.where(np.isfinite(x[r][t]), np.abs(x[r][t] - x[r][t].max()), 0) + (E / 8 + 8) + 4
                part[t] += s * np.abs((gg * p).sum()) * rel
        bound = 1.01 * 2 * U * part + HALF[dtype] * np.abs(want[r]) + TINY[dtype]
        near(f64(d)[r], want[r], bound, f"d_logits of rank {r}")


ROUTES = [
    # ranks, tokens, E, K, options
    (1, [1], 1, 1, dict()),
    (2, [3, 0], 5, 5, dict(score="sigmoid")),
    (3, [7, 1, 40], 8, 2, dict(renormalize=False)),
    (4, [33, 0, 2, 65], 60, 6, dict(score="sigmoid", renormalize=False, scale=2.5)),
    (8, [9] * 8, 256, 8, dict(score="sigmoid", bias=True, groups=8, top_groups=4, scale=2.5)),
    (2, [50, 21], 256, 8, dict(score="softmax", bias=True, groups=8, top_groups=3, group_by="max")),
    (2, [31, 64], 160, 6, dict(score="softmax", groups=8, top_groups=3, group_by="max", renormalize=False)),
    (1, [70], 160, 6, dict(score="softmax", groups=8, top_groups=3, group_by="top2")),
    (2, [5, 6], 257, 9, dict(score="softmax")),
    (1, [17], 512, 10, dict(score="softmax", bias=True)),
    (1, [9], 1024, 16, dict(score="sigmoid", bias=True)),
    (1, [9], 1000, 16, dict(score="softmax", groups=40, top_groups=7)),
    (1, [9], 64, 16, dict(score="sigmoid", groups=64, top_groups=20)),
    (1, [12], 1023, 12, dict(score="sigmoid", groups=33, top_groups=4, bias=True)),
    (16, [3] * 16, 48, 3, dict(score="sigmoid", groups=3, top_groups=2, group_by="top2", bias=True)),
    (2, [11, 13], 36, 4, dict(groups=12, top_groups=4, group_by="top2", bias=True)),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(ROUTES)))
def test_route_and_gradient(case, dtype):
    R, tokens, E, K, kw = ROUTES[case]
    kw = dict(kw)
    g = gen(100 + case)
    logits = [normal(g, t, E, std=2.0, dtype=dtype) for t in tokens]
    for l in logits:  # some experts masked out, some rows altogether, some almost
        l[torch.rand(l.shape, generator=g) < 0.1] = -math.inf
        if l.shape[0] > 2:
            l[1] = -math.inf
            l[2, 1:] = -math.inf
    if kw.get("bias"):
        kw["bias"] = normal(g, E, std=0.1)
    _, e = check_route(logits, K, dtype, **kw)
    check_route_grad(logits, [x.cpu() for x in e], dtype, kw.get("score", "softmax"), kw.get("renormalize", True),
                     kw.get("scale", 1.0), 300 + case)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", ["none", "zeros", "steps"])
def test_route_ties_go_to_the_lower_index(dtype, score, bias):
    g = gen(9)
    E = 64
    logits = [torch.randint(-2, 3, (40, E), generator=g).to(TYPES[dtype]), torch.zeros(3, E, dtype=TYPES[dtype])]
    logits[1][1] = -0.0
    logits[1][2, ::2] = -0.0  # zeros of both signs are one value
    b = {"none": None, "zeros": torch.zeros(E), "steps": torch.arange(E).float() % 2}[bias]
    for kw in (dict(), dict(groups=8, top_groups=2, group_by="max"), dict(groups=8, top_groups=2, group_by="top2")):
        check_route(logits, 8, dtype, score=score, bias=b, **kw)


def test_route_tells_close_scores_apart():
    """Scores that agree in float32: sigmoids near one, and logits one step
    apart under a bias; the choice is by the 64-bit value."""
    E = 16
    l = torch.linspace(17.0, 20.0, E).view(1, E).contiguous()
    check_route([l], 4, "f32", score="sigmoid", bias=torch.zeros(E))
    check_route([l], 4, "f32", score="sigmoid")
    step = torch.full((1, E), 0.3)
    for j in range(E):
        step[0, j] = float(np.nextafter(np.float32(0.3), np.float32(1))) if j % 3 == 0 else 0.3
    check_route([step], 7, "f32", score="sigmoid", bias=torch.full((E,), 0.25))
    check_route([step], 7, "f32", score="softmax", bias=torch.full((E,), 0.25))
    check_route([step], 7, "f32", score="softmax", groups=4, top_groups=2, group_by="top2")
    # near 18 a step of the logits moves the sigmoid by 3e-14: hundreds of steps of
    # a double, a fraction of one of its upper 42 bits
    fine = torch.full((1, E), 18.0) + 2.0 ** -19 * torch.randperm(E, generator=gen(3)).float()
    for b in (0.0, 0.25, -0.5):
        check_route([fine], 5, "f32", score="sigmoid", bias=torch.full((E,), b))
        check_route([fine], 5, "f32", score="sigmoid", bias=torch.full((E,), b), groups=4, top_groups=3)


@pytest.mark.parametrize("K", [2, 4, 8, 16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_close_scores_in_one_group(K, score):
    """All chosen experts, and the next one close behind, in one group of those
    that are far apart: the last place goes by what float32 does not tell."""
    g = gen(13)
    E, size = 100, 20
    for _ in range(2):
        l = torch.full((6, E), -4.0)
        l[:, 60:80] = torch.linspace(2.0, 0.0, size)[torch.argsort(torch.rand(6, size, generator=g), 1)]
        for t in range(6):
            rank = torch.argsort(l[t, 60:80], descending=True) + 60
            l[t, rank[K]] = l[t, rank[K - 1]]  # the bias decides
        # few tokens, and enough for a lane to have a group of its own
        check_route([l, l.repeat(350, 1)], K, "f32", score=score, bias=torch.rand(E, generator=g) * 2.0 ** -28, groups=5,
                    top_groups=1)
    # and by what the upper 42 bits of the scores do not
    fine = torch.full((6, E), 15.0)
    for t in range(6):
        fine[t, 60:80] = 18.0 + 2.0 ** -19 * torch.randperm(size, generator=g).float()
    for b in (0.0, 0.25):
        check_route([fine, fine.repeat(350, 1)], K, "f32", score="sigmoid", bias=torch.full((E,), b), groups=5, top_groups=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_extreme_logits(score, groups):
    """NaN, infinities and the type's lowest values."""
    g = gen(11)
    E = 32
    l = normal(g, 8, E, std=3.0)
    l[0, 3] = math.nan
    l[1, 5] = math.inf
    l[2] = torch.finfo(torch.float32).min
    l[3, ::2] = torch.finfo(torch.float32).min
    l[4] = -math.inf
    l[4, 7] = 1.0
    l[5] = math.nan
    l[6, :] = 80.0
    l[7] = -60.0
    for bias in (None, normal(g, E, std=0.1)):
        _, e = check_route([l], 4, "f32", score=score, bias=bias, groups=groups, top_groups=min(2, groups),
                           renormalize=False)
        _, e = check_route([l], 4, "f32", score=score, bias=bias, groups=groups, top_groups=min(2, groups))
    e = e[0].cpu()
    assert e[5].tolist() == [-1] * 4
    if score == "softmax":
        assert e[0].tolist() == [-1] * 4 and e[1].tolist() == [-1] * 4
    b = torch.zeros(E)
    b[::2] = -math.inf
    b[1] = math.nan
    check_route([l], 16, "f32", score=score, bias=b, groups=1)


def test_route_unaligned_rows_and_outputs():
    g = gen(12)
    for dtype in ("f32", "bf16"):
        logits = [normal(g, 9, 64, dtype=dtype), normal(g, 4, 64, dtype=dtype)]
        l = shifted(dev(logits), 1)
        with session(2):
            w, e = rr.route(l, 6)
            w2, e2 = rr.route(dev(logits), 6)
            d = rr.route_grad(l, e, w, out=shifted([torch.zeros_like(x) for x in l], 3))
            d2 = rr.route_grad(dev(logits), e2, w2)
            torch.cuda.synchronize()
        for a, b in zip(w + e + d, w2 + e2 + d2):
            assert torch.equal(a, b)


def test_route_gradient_with_repeated_and_foreign_experts():
    """A gradient call may name an expert twice or none: parts add up, indices
    outside the experts have none."""
    l = normal(gen(13), 2, 12)
    e = torch.tensor([[3, 3, 5], [-1, 400, 2]], dtype=torch.int32)
    for score in ("softmax", "sigmoid"):
        with session(1):
            dw = torch.tensor([[1.0, 2.0, 4.0], [7.0, 9.0, 3.0]])
            d = rr.route_grad([l.to(DEV)], [e.to(DEV)], [dw.to(DEV)], score=score, renormalize=False)[0].cpu()
        want = orc.route_grad(f64([l]), [e.numpy()], f64([dw]), score=score, renormalize=False)[0]
        near(d.double().numpy(), want, 64 * U * (np.abs(want) + 8), score)


# ---------------------------------------------------------------- dispatch and combine

def choices(g, tokens, E, K, none=0.1):
    out = []
    for t in tokens:
        pop = torch.randn(E, generator=g) * 0.7
        e = torch.argsort(torch.randn(t, E, generator=g) + pop, dim=1)[:, :K].to(torch.int32)
        e[torch.rand(t, K, generator=g) < none] = -1
        out.append(e.contiguous())
    return out


def check_plan(experts, E, capacity):
    """The plan against the oracle; returns it, in an open session."""
    plan = rr.dispatch_plan(dev(experts), E, capacity=capacity)
    torch.cuda.synchronize()
    caps = plan.capacity
    slots, offsets, counts = orc.dispatch_plan(ints(experts), E, caps)
    for r in range(len(experts)):
        assert np.array_equal(ints(plan.slots)[r], slots[r]), f"slots of rank {r}"
        assert np.array_equal(ints(plan.offsets)[r], offsets[r]), f"offsets of rank {r}"
        assert np.array_equal(ints(plan.counts)[r], counts[r]), f"counts of rank {r}"
    return plan


PLANS = [
    # ranks, tokens, E, K, capacity
    (1, [0], 1, 1, None),
    (1, [1], 1, 1, None),
    (2, [5, 0], 4, 3, 2),
    (4, [33, 0, 17, 64], 12, 4, 40),
    (8, [8] * 8, 64, 8, None),
    (16, [7] * 16, 1024, 16, 3),
    (3, [700, 1, 500], 9, 2, [100, 0, 5000]),
    (2, [1024, 1000], 6, 6, None),      # over one workgroup's entries
    (4, [4096, 1, 0, 2500], 128, 4, 3000),
    (5, [0, 0, 9000, 0, 3], 1000, 3, None),
]


@pytest.mark.parametrize("case", range(len(PLANS)))
def test_plan(case):
    R, tokens, E, K, capacity = PLANS[case]
    with session(R):
        check_plan(choices(gen(400 + case), tokens, E, K), E, capacity)


def test_plan_of_one_expert_and_of_foreign_ones():
    with session(2):
        e = [torch.full((3000, 4), 1, dtype=torch.int32), torch.full((50, 4), -7, dtype=torch.int32)]
        check_plan(e, 2, None)
        e = [torch.full((30, 4), 2, dtype=torch.int32), torch.full((5, 4), 2**31 - 1, dtype=torch.int32)]
        plan = rr.dispatch_plan(dev(e), 2)
        torch.cuda.synchronize()
        assert all((s == -1).all() for s in plan.slots) and not any(c.any() for c in plan.counts)


MOVES = [
    # ranks, tokens, E, K, capacity, width
    (1, [1], 1, 1, None, 1),
    (2, [3, 0], 4, 2, None, 7),
    (4, [9, 1, 0, 20], 8, 3, 12, 64),
    (3, [5, 6, 7], 6, 6, None, 257),
    (8, [4] * 8, 64, 8, None, 1024),
    (2, [40, 41], 16, 16, None, 130),
    (2, [3, 2], 32, 10, None, 5000),
    (16, [2] * 16, 16, 4, 5, 33),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(MOVES)))
@pytest.mark.parametrize("off", [0, 1])
def test_dispatch_and_combine(case, dtype, off):
    R, tokens, E, K, capacity, D = MOVES[case]
    g = gen(500 + case)
    ex = choices(g, tokens, E, K)
    xs = [normal(g, t, D, dtype=dtype) for t in tokens]
    weights = [torch.rand(t, K, generator=g) for t in tokens]
    d_outs = [normal(g, t, D, dtype=dtype) for t in tokens]
    h = HALF[dtype]
    with session(R):
        plan = check_plan(ex, E, capacity)
        mark = -776.0  # a value of every type
        fresh = lambda: shifted([torch.full((c, D), mark, dtype=TYPES[dtype], device=DEV) for c in plan.capacity], off)
        rows = rr.dispatch(shifted(dev(xs), off), plan, out=fresh())
        slots = ints(plan.slots)
        exn = ints(ex)
        want = orc.dispatch(f64(xs), exn, slots, E, [np.full((c, D), mark) for c in plan.capacity])
        for d in range(R):
            assert np.array_equal(f64(rows)[d], want[d]), f"rows of rank {d}"
        filled = [normal(g, c, D, dtype=dtype) for c in plan.capacity]
        frows = shifted(dev(filled), off)
        for w in (weights, None):
            got = rr.combine(frows, plan, None if w is None else dev(w), out=shifted([torch.zeros_like(x) for x in dev(xs)], off))
            torch.cuda.synchronize()
            want, size = orc.combine(f64(filled), exn, slots, E, None if w is None else f64(w))
            for r in range(R):
                near(f64(got)[r], want[r], 1.01 * (K + 1) * U * size[r] + h * np.abs(want[r]) + TINY[dtype], f"combined rank {r}")
        dr, dw = rr.combine_grad(shifted(dev(d_outs), off), frows, plan, dev(weights),
                                 out=(fresh(), [torch.full_like(w, mark) for w in dev(weights)]))
        torch.cuda.synchronize()
    want_r, want_w, size = orc.combine_grad(f64(d_outs), f64(filled), exn, slots, E, f64(weights),
                                            [np.full((c, D), mark) for c in plan.capacity])
    # products in float32, one chain of D/256 per lane (16-byte vectors) and two trees
    chain = math.ceil(D / 256) + 16 + 10
    for r in range(R):
        near(f64(dr)[r], want_r[r], 1.01 * U * np.abs(want_r[r]) + h * np.abs(want_r[r]) + TINY[dtype], f"d_rows of rank {r}")
        near(f64(dw)[r], want_w[r], 1.01 * chain * U * size[r] + 2.0 ** -149, f"d_weights of rank {r}")


def test_moves_never_follow_foreign_indices():
    """Slots and experts out of range count as none, in every call."""
    R, E, K, D = 2, 4, 2, 16
    with session(R):
        ex = [torch.tensor([[0, 3], [-5, 2]], dtype=torch.int32), torch.tensor([[2**31 - 1, 1]], dtype=torch.int32)]
        plan = rr.dispatch_plan(dev(ex), E, capacity=3)
        for s, v in zip(plan.slots, ([[0, 3], [1, -2**31]], [[1, 2**31 - 1]])):
            s.copy_(torch.tensor(v, dtype=torch.int32))
        xs = [torch.ones(2, D, device=DEV), torch.full((1, D), 2.0, device=DEV)]
        rows = rr.dispatch(xs, plan)
        torch.cuda.synchronize()
        assert torch.equal(rows[0][0], xs[0][0]) and float(sum(r.sum() for r in rows)) == D
        ys = rr.combine([torch.ones(3, D, device=DEV)] * 2, plan)
        dr, dw = rr.combine_grad(ys, rows, plan, [torch.ones(2, K, device=DEV), torch.ones(1, K, device=DEV)])
        torch.cuda.synchronize()
        assert ys[0][0].sum() == D and not ys[0][1].any() and not ys[1].any()
        assert dw[0].cpu().tolist() == [[D, 0], [0, 0]] and dw[1].cpu().tolist() == [[0, 0]]
        assert float(sum(r.sum() for r in dr)) == D


def test_combine_skips_what_has_no_slot():
    """Rows behind the last entry may hold NaN, and so may weights of empty slots."""
    with session(1):
        ex = [torch.tensor([[0, -1], [-1, -1]], dtype=torch.int32)]
        plan = rr.dispatch_plan(dev(ex), 1)
        rows = [torch.full((4, 8), math.nan, device=DEV)]
        rows[0][0] = 3.0
        w = [torch.tensor([[2.0, math.nan], [math.nan, math.inf]], device=DEV)]
        y = rr.combine(rows, plan, w)[0].cpu()
        dr, dw = rr.combine_grad([torch.ones(2, 8, device=DEV)], rows, plan, w)
        assert torch.equal(y, torch.tensor([[6.0] * 8, [0.0] * 8]))
        assert dw[0].cpu().tolist() == [[24.0, 0.0], [0.0, 0.0]]
        assert torch.equal(dr[0].cpu(), torch.tensor([[2.0] * 8] + [[0.0] * 8] * 3))


# ---------------------------------------------------------------- embedding

def token_ids(g, tokens, vocab, id_type, none=0.1):
    out = []
    for t in tokens:
        u = torch.rand(t, generator=g, dtype=torch.float64)
        i = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
        i[torch.rand(t, generator=g) < none] = -1
        out.append(i.to(id_type))
    return out


EMBEDS = [
    # ranks, tokens, vocab, width, scale
    (1, [1], 1, 1, 1.0),
    (2, [0, 0], 3, 5, 2.0),
    (2, [63, 1], 11, 64, 1.0),
    (4, [64, 0, 65, 3], 5, 130, 0.3),
    (3, [200, 128, 1], 100, 257, 22.6),
    (8, [40] * 8, 1031, 33, 1.0),
    (4, [2100, 0, 5000, 1500], 700, 24, 0.125),   # over one workgroup's ids
    (2, [9000, 400], 70001, 8, 1.5),              # several blocks, two digits
    (16, [17] * 16, 40, 2056, 1.0),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("case", range(len(EMBEDS)))
@pytest.mark.parametrize("off", [0, 1])
def test_embedding_and_gradient(case, dtype, off):
    R, tokens, V, D, scale = EMBEDS[case]
    g = gen(600 + case)
    id_type = torch.int64 if case % 2 else torch.int32
    ids = token_ids(g, tokens, V, id_type)
    table = normal(g, V, D, dtype=dtype)
    bounds = orc.shard_bounds(V, R)
    d_outs = [normal(g, t, D, dtype=dtype) for t in tokens]
    h = HALF[dtype]
    with session(R):
        shards = shifted([table[lo:hi].to(DEV) for lo, hi in bounds], off)
        got = rr.embedding(dev(ids), shards, scale=scale, out=shifted([torch.full_like(x, 9.0) for x in dev(d_outs)], off))
        torch.cuda.synchronize()
        want = orc.embedding(ints(ids), table.double().numpy(), float(np.float32(scale)))
        for r in range(R):
            near(f64(got)[r], want[r], (0 if scale == 1.0 else 1.01 * U + h) * np.abs(want[r]) + (scale != 1.0) * TINY[dtype],
                 f"looked up, rank {r}")
        exact, size, count = orc.embedding_grad(ints(ids), f64(d_outs), V, float(np.float32(scale)))
        depth = np.minimum(count, 64) + np.minimum(-(-count // 64), 16) + -(-count // 1024) + 2
        for out_type in {"f32", dtype}:
            for accumulate in (False, True):
                held = [normal(g, hi - lo, D, dtype=out_type) for lo, hi in bounds]
                out = shifted(dev(held), off)
                rr.embedding_grad(dev(ids), shifted(dev(d_outs), off), V, scale=scale, out=out, accumulate=accumulate)
                torch.cuda.synchronize()
                full = np.concatenate(f64(out))
                old = torch.cat(held).double().numpy()
                ordered = orc.embedding_grad_ordered(ints(ids), f64(d_outs), V, scale, old if accumulate else None)
                want = torch.from_numpy(ordered).to(TYPES[out_type]).double().numpy()
                assert np.array_equal(full, want), f"gradient in {out_type}, accumulate {accumulate}"
                true = exact + (old if accumulate else 0)
                bound = 1.01 * depth[:, None] * U * (size + (np.abs(old) if accumulate else 0)) + \
                    HALF[out_type] * np.abs(true) + TINY[out_type]
                near(full, true, bound, "gradient against 64 bits")


@pytest.mark.parametrize("counts", [
    [64], [65], [63, 65, 64], [128, 1, 129], [1] * 63 + [200], [64] * 5, [10, 4096], [4097, 3], [1, 9000, 2],
    [70, 70, 70, 1, 1, 130], [62, 1, 1, 128, 127], [5000, 5000],
])
@pytest.mark.parametrize("ranks", [1, 3])
def test_embedding_grad_long_sums(counts, ranks):
    """Ids with as many tokens as a piece, a run of pieces, and around them, at
    every position of a window; with and without ids outside the table."""
    g = gen(sum(counts))
    ids = torch.cat([torch.full((c,), v) for v, c in enumerate(counts)] + [torch.full((37,), -1)])
    ids = ids[torch.randperm(ids.numel(), generator=g)]
    parts = list(ids.to(torch.int32).split(-(-ids.numel() // ranks)))
    parts += [ids[:0].to(torch.int32)] * (ranks - len(parts))
    D, V = 12, len(counts) + 2
    d_outs = [normal(g, p.numel(), D) for p in parts]
    with session(ranks):
        out = rr.embedding_grad(dev(parts), dev(d_outs), V, scale=3.0)
        torch.cuda.synchronize()
    want = orc.embedding_grad_ordered(ints(parts), f64(d_outs), V, 3.0)
    assert np.array_equal(np.concatenate(f64(out)), want.astype(np.float64))


@pytest.mark.parametrize("vocab", [5, 4096, 4097, 300001])
@pytest.mark.parametrize("n", [64, 65, 1025, 4097, 8191, 8192, 8193])
def test_embedding_grad_sorts(n, vocab):
    """Around what one launch sorts, and the table rows it marks at a time."""
    g = gen(n + vocab)
    ids = token_ids(g, [n // 3, n - n // 3], vocab, torch.int64)
    ids[1][-1] = vocab - 1
    d_outs = [normal(g, i.numel(), 3) for i in ids]
    with session(2):
        out = rr.embedding_grad(dev(ids), dev(d_outs), vocab)
        torch.cuda.synchronize()
    want = orc.embedding_grad_ordered(ints(ids), f64(d_outs), vocab, 1.0)
    assert np.array_equal(np.concatenate(f64(out)), want.astype(np.float64))


def test_embedding_passes_special_values_through():
    with session(1):
        bits = torch.tensor([0x7FC1, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x7F7F, 0x3F80, 0x8001], dtype=torch.int32)
        table = bits.to(torch.int16).view(torch.bfloat16).view(1, 8).to(DEV)
        y = rr.embedding([torch.zeros(2, dtype=torch.int64, device=DEV)], [table])[0]
        assert torch.equal(y.view(torch.int16).cpu(), bits.to(torch.int16).repeat(2, 1))
        big = torch.tensor([2**33, -2**33, 0, 2**31], dtype=torch.int64, device=DEV)  # ids past 32 bits
        y = rr.embedding([big], [torch.ones(5, 8, device=DEV)])[0].cpu()
        assert y.sum(1).tolist() == [0, 0, 8, 0]
        d = rr.embedding_grad([big], [torch.ones(4, 8, device=DEV)], 5)[0].cpu()
        assert d.sum(1).tolist() == [8, 0, 0, 0, 0]


def test_embedding_without_tokens_clears_the_gradient():
    with session(2):
        none = [torch.zeros(0, dtype=torch.int32, device=DEV)] * 2
        d = [torch.zeros(0, 6, device=DEV)] * 2
        out = [torch.full((3, 6), 5.0, device=DEV), torch.full((2, 6), 5.0, device=DEV)]
        rr.embedding_grad(none, d, 5, out=out, accumulate=True)
        torch.cuda.synchronize()
        assert all((o == 5.0).all() for o in out)
        rr.embedding_grad(none, d, 5, out=out)
        torch.cuda.synchronize()
        assert not any(o.any() for o in out)


# ---------------------------------------------------------------- together

def layer_reference(x, table, wr, we, bias, ids, K, groups, top_groups):
    """One expert layer on one token batch, differentiable, in 64 bits on the CPU."""
    h = table[ids]
    s = torch.sigmoid(h @ wr)
    with torch.no_grad():
        _, e = orc.route([(h @ wr).numpy()], K, score="sigmoid", bias=bias.numpy(), groups=groups, top_groups=top_groups)
        e = torch.from_numpy(e[0]).long()
    w = torch.gather(s, 1, e)
    w = 2.5 * w / w.sum(1, keepdim=True)
    y = torch.stack([sum(w[t, k] * torch.tanh(h[t] * we[e[t, k]]) for k in range(K)) for t in range(h.shape[0])])
    return y


def test_an_expert_layer_forward_and_backward():
    """Embedding, router, dispatch, elementwise experts, combine, and all the
    gradients back into the sharded table and the router, against autograd in
    64 bits on the CPU.  Bound: 2^-24 times the roundings in a chain (the
    longest: ~60 through router product, weights, combine and table sums),
    taken 4 times for the products they pass through, of the largest value."""
    R, T, V, D, E, K = 4, 12, 50, 16, 8, 3
    g = gen(77)
    table = normal(g, V, D).double().requires_grad_()
    wr = (normal(g, D, E) * 0.5).double().requires_grad_()
    we = normal(g, E, D).double().requires_grad_()
    bias = normal(g, E, std=0.1)
    ids = [torch.randint(0, V, (T,), generator=g) for _ in range(R)]
    dy = [normal(g, T, D) for _ in range(R)]
    want = layer_reference(None, table, wr, we, bias.double(), torch.cat(ids), K, 4, 2)
    (want * torch.cat(dy).double()).sum().backward()

    kw = dict(score="sigmoid", renormalize=True, scale=2.5)
    per = E // R
    with session(R):
        shards = [table.detach().float()[lo:hi].contiguous().to(DEV) for lo, hi in orc.shard_bounds(V, R)]
        wrd, wed = wr.detach().float().to(DEV), we.detach().float().to(DEV)
        idd, dyd = dev(ids), dev(dy)
        h = rr.embedding(idd, shards)
        logits = [x @ wrd for x in h]
        w, e = rr.route(logits, K, bias=bias.to(DEV), groups=4, top_groups=2, **kw)
        plan = rr.dispatch_plan(e, E)
        rows = rr.dispatch(h, plan)
        # each row's expert, from the offsets
        which = [torch.bucketize(torch.arange(c, device=DEV), o[1:], right=True).clamp(max=per - 1)
                 for c, o in zip(plan.capacity, plan.offsets)]
        inner = [r * wed[d * per + i] for d, (r, i) in enumerate(zip(rows, which))]
        results = [torch.tanh(x) for x in inner]
        y = rr.combine(results, plan, w)
        d_results, d_w = rr.combine_grad(dyd, results, plan, w)
        d_inner = [dr * (1 - r * r) for dr, r in zip(d_results, results)]
        d_rows = [di * wed[d * per + i] for d, (di, i) in enumerate(zip(d_inner, which))]
        d_h = rr.combine(d_rows, plan)
        d_logits = rr.route_grad(logits, e, d_w, **kw)
        d_h = [a + b @ wrd.t() for a, b in zip(d_h, d_logits)]
        d_table = rr.embedding_grad(idd, d_h, V)
        d_wr = sum(x.t() @ b for x, b in zip(h, d_logits))
        torch.cuda.synchronize()

    def close(got, ref, what):
        near(got.detach().cpu().double().numpy(), ref.detach().numpy(),
             np.full(ref.shape, 4 * 60 * U * float(ref.detach().abs().max())), what)

    close(torch.cat(y), want, "output")
    close(torch.cat(d_table), table.grad, "d_table")
    close(d_wr, wr.grad, "d_router")


def moe_inputs(seed, R=3, T=41, V=300, D=72, E=12, K=2, dtype="bf16"):
    g = gen(seed)
    return dict(ids=token_ids(g, [T] * R, V, torch.int64), table=normal(g, V, D, dtype=dtype),
                logits=[normal(g, T, E) for _ in range(R)], dy=[normal(g, T, D, dtype=dtype) for _ in range(R)])


def moe_chain(st):
    """All entry points in a row; everything allocated on the way."""
    h = rr.embedding(st["ids"], st["shards"], scale=2.0)
    w, e = rr.route(st["logits"], 2, score="sigmoid")
    plan = rr.dispatch_plan(e, 12, capacity=60)
    rows = rr.dispatch(h, plan)
    y = rr.combine(rows, plan, w)
    dr, dw = rr.combine_grad(st["dy"], rows, plan, w)
    dh = rr.combine(dr, plan)
    dl = rr.route_grad(st["logits"], e, dw, score="sigmoid")
    dt = rr.embedding_grad(st["ids"], dh, 300, scale=2.0, dtype=torch.float32)
    return w + e + plan.slots + plan.offsets + plan.counts + rows + y + dr + dw + dl + dt


def moe_state(seed):
    i = moe_inputs(seed)
    return dict(ids=dev(i["ids"]), logits=dev(i["logits"]), dy=dev(i["dy"]),
                shards=[i["table"][lo:hi].contiguous().to(DEV) for lo, hi in orc.shard_bounds(300, 3)])


def test_results_do_not_change_between_runs():
    with session(3):
        st = moe_state(1)
        first = [t.clone() for t in moe_chain(st)]
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, moe_chain(st)))


def test_two_captured_graphs_share_nothing():
    """Two chains captured into graphs of their own, replayed several times
    with fresh inputs, eager work in between, in turn and on two streams at
    once, each against the eager results."""
    with session(3):
        states = [moe_state(2), moe_state(3)]
        for st in states:
            moe_chain(st)
        torch.cuda.synchronize()
        graphs, outs = [], []
        for st in states:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(moe_chain(st))
            graphs.append(graph)
        streams = [torch.cuda.Stream() for _ in graphs]
        for rep in range(4):
            for n, st in enumerate(states):
                new = moe_state(10 * rep + n + 20)
                for key in st:
                    for a, b in zip(st[key], new[key]):
                        a.copy_(b)
            want = [[t.clone() for t in moe_chain(st)] for st in states]
            torch.cuda.synchronize()
            for graph, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
            torch.cuda.synchronize()
            for got, ref in zip(outs, want):
                assert all(torch.equal(a, b) for a, b in zip(got, ref)), f"replay {rep}"


def test_other_streams():
    """Calls on a side stream, by the stream argument and as the current one,
    ordered behind the work that makes their inputs there."""
    with session(3):
        want = [t.clone() for t in moe_chain(moe_state(4))]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = moe_chain(moe_state(4))
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        st = moe_state(4)
        s.wait_stream(torch.cuda.current_stream())
        w, e = rr.route(st["logits"], 2, score="sigmoid", stream=s)
        plan = rr.dispatch_plan(e, 12, capacity=60, stream=s.cuda_stream)
        h = rr.embedding(st["ids"], st["shards"], scale=2.0, stream=s)
        rows = rr.dispatch(h, plan, stream=s)
        y = rr.combine(rows, plan, w, stream=s)
        s.synchronize()
        got = w + e + plan.slots + plan.offsets + plan.counts + rows + y
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_tensors_elsewhere_are_refused():
    with session(2):
        cpu = [torch.zeros(2, 4), torch.zeros(2, 4)]
        with pytest.raises(ValueError):
            rr.route(cpu, 1)
        with pytest.raises(rr.CollectiveError):
            rr.route([torch.zeros(2, 4, device=DEV), torch.zeros(2, 4)], 1)
        with pytest.raises(rr.CollectiveError):
            rr.route([torch.zeros(2, 4, device=DEV)] * 3, 1)


# ---------------------------------------------------------------- large buffers, calls at once

# Rows beyond 2^31 elements (2^32 bytes in bf16) of one buffer: results there are
# those of the same rows in small buffers, bit for bit.
FAR = 2 ** 31 // 4096 + 9  # rows of 4096


def test_far_route_rows():
    with session(2):
        few = normal(gen(1), 3, 1024, dtype="bf16").to(DEV)
        many = torch.zeros(2 ** 21 + 5, 1024, dtype=torch.bfloat16, device=DEV)
        many[-3:] = few
        dw = torch.zeros(many.shape[0], 4, device=DEV)
        dw[-3:] = normal(gen(2), 3, 4).to(DEV)
        none = [few[:0], dw[:0]]
        w, e = rr.route([none[0], many], 4)
        ws, es = rr.route([none[0], few], 4)
        assert torch.equal(w[1][-3:], ws[1]) and torch.equal(e[1][-3:], es[1])
        d = rr.route_grad([none[0], many], e, [none[1], dw])
        ds = rr.route_grad([none[0], few], es, [none[1], dw[-3:].clone()])
        assert torch.equal(d[1][-3:], ds[1])
        assert not d[1][:-3].any()


def test_far_exchanged_rows():
    """One expert on rank 1 takes every token of rank 0."""
    with session(2):
        x = torch.zeros(FAR, 4096, dtype=torch.bfloat16, device=DEV)
        x[-8:] = normal(gen(3), 8, 4096, dtype="bf16").to(DEV)
        none = x[:0]
        e = torch.ones(FAR, 1, dtype=torch.int32, device=DEV)
        plan = rr.dispatch_plan([e, e[:0]], 2, capacity=[0, FAR])
        assert torch.equal(plan.slots[0][:, 0], torch.arange(FAR, dtype=torch.int32, device=DEV))
        rows = rr.dispatch([x, none], plan)
        assert torch.equal(rows[1], x)
        half = torch.full((FAR, 1), 0.5, device=DEV)
        y = rr.combine(rows, plan, [half, half[:0]])[0]
        assert torch.equal(y[-8:], x[-8:] * 0.5) and not y[:-8].any()
        del y
        dx, dw = rr.combine_grad([x, none], rows, plan, [half, half[:0]])
        assert torch.equal(dx[1][-8:], x[-8:] * 0.5) and not dx[1][:-8].any()
        want = (f64([x[-8:]])[0] ** 2).sum(1)
        near(dw[0][-8:, 0].cpu().numpy(), want, 1.01 * 4096 * U * want, "d_weights")


def test_far_table_rows_and_tokens():
    with session(2):
        vocab = 2 * FAR
        tables = [torch.zeros(FAR, 4096, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        tables[1][-8:] = normal(gen(4), 8, 4096, dtype="bf16").to(DEV)
        ids = torch.full((FAR,), -1, dtype=torch.int64, device=DEV)
        ids[-12:-4] = torch.arange(vocab - 8, vocab)
        ids[-4:] = vocab - 1
        none = ids[:0]
        y = rr.embedding([ids, none], tables)[0]
        assert torch.equal(y[-12:-4], tables[1][-8:]) and torch.equal(y[-4:], tables[1][-1:].expand(4, -1))
        assert not y[:-12].any()
        d = rr.embedding_grad([ids, none], [y, y[:0]], vocab)
        got, near_rows = d[1][-8:], rr.embedding_grad([ids[-12:], none], [y[-12:].clone(), y[:0]], vocab)[1][-8:]
        assert torch.equal(got, near_rows)
        assert torch.equal(got[:-1], tables[1][-8:-1])
        assert not d[0].any() and not d[1][:-8].any()


def test_calls_from_two_threads_at_once():
    """Two threads, a stream each, the whole chain several times."""
    with session(3):
        states = [moe_state(5), moe_state(6)]
        want = [[t.clone() for t in moe_chain(st)] for st in states]
        torch.cuda.synchronize()
        wrong = []

        def work(n):
            with torch.cuda.stream(torch.cuda.Stream()):
                for rep in range(5):
                    got = moe_chain(states[n])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                        wrong.append((n, rep))

        threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not wrong


def test_small_outputs_share_an_allocation_and_large_ones_do_not():
    with session(3):
        e = [torch.zeros(4, 1, dtype=torch.int32, device=DEV)] * 3
        for width, together in ((40, True), (2 ** 20 + 8, False)):
            xs = [normal(gen(7), 4, width, dtype="bf16").to(DEV) for _ in range(3)]
            plan = rr.dispatch_plan(e, 3, capacity=[12, 1, 5])
            rows = rr.dispatch(xs, plan)
            assert [tuple(x.shape) for x in rows] == [(12, width), (1, width), (5, width)]
            assert torch.equal(rows[0], torch.cat(xs)) and not rows[1].any() and not rows[2].any()
            assert all(x.data_ptr() % 256 == 0 for x in rows)
            stores = {x.untyped_storage().data_ptr() for x in rows}
            assert len(stores) == (1 if together else 3)
            rows[1].fill_(3)  # each is a tensor of its own
            assert torch.equal(rows[0], torch.cat(xs)) and not rows[2].any()
