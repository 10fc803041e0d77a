"""Row exchanges on the GPU where scores saturate, one expert outweighs all
others, rows are masked out and sums leave float32's range.

u = 2^-24 is float32's half step.  References are computed in 64 bits.
"""

import math

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


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------- the order where scores saturate

def saturated_rows(score, E, g):
    """Rows of logits whose scores in 64 bits are exactly alike, however exp
    rounds: sigmoids of one and of zero, softmax scores of zero, and logits too
    small to move either; smaller logits at lower indices among them."""
    def shuffled(v):
        return v[torch.randperm(E, generator=g)]

    up, plain = torch.arange(E).float(), torch.randn(E, generator=g)
    far = 2.0 ** -70 * (up + 1)
    few = plain.clone()
    few[[1, 4, E - 2]] = torch.tensor([41.0, 47.0, 44.0])
    masked = plain.clone()
    masked[E // 3:] = shuffled(-1e4 - 16 * up)[E // 3:]
    most = torch.full((E,), -1e4)
    most[[2, E - 1]] = torch.tensor([1.0, -9e3])
    most[1::2] -= 512
    rows = [shuffled(-900.0 - up), masked, most, shuffled(far), shuffled(-far), shuffled(far - 2.0 ** -70 * E / 2),
            torch.where(shuffled(up) < E / 2, shuffled(far), -3.0), torch.zeros(E), few]
    if score == "sigmoid":
        rows += [40.0 + up, shuffled(40.0 + up), torch.where(up % 3 == 0, 60 - up / E, -800.0 - up)]
    else:
        rows += [torch.where(shuffled(up) < 3, 5.0, shuffled(far)), torch.where(shuffled(up) < 1, 900.0, plain),
                 torch.where(shuffled(up) < 2, 900.0, shuffled(far))]
    return torch.stack(rows)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,groups,top_groups,group_by", [
    (12, 4, 1, 1, "max"), (60, 16, 1, 1, "max"), (256, 8, 1, 1, "max"), (320, 8, 1, 1, "max"),
    (32, 4, 4, 2, "max"), (256, 8, 8, 3, "max"), (256, 8, 8, 3, "top2"), (60, 5, 12, 4, "max"), (40, 3, 40, 6, "top2"),
])
def test_saturated_scores_go_to_the_lower_index(dtype, score, E, K, groups, top_groups, group_by):
    """With no bias and with one of zeros, few tokens and many."""
    l = saturated_rows(score, E, gen(E + K)).to(TYPES[dtype])
    kw = dict(score=score, groups=groups, top_groups=top_groups, group_by=group_by)
    _, want = orc.route([l.double().numpy()], K, **kw)
    times = 200
    with session(1):
        for bias in (None, torch.zeros(E, device=DEV)):
            for reps in (1, times):
                _, e = rr.route([l.repeat(reps, 1).to(DEV)], K, bias=bias, **kw)
                e = e[0].cpu().numpy().reshape(reps, *want[0].shape)
                for t in range(want[0].shape[0]):
                    assert (e[:, t] == want[0][t]).all(), \
                        f"bias {bias is not None}, {reps} times, row {t}: {e[0, t]} not {want[0][t]}"


def test_neighbouring_logits_with_one_sigmoid():
    """Steps of a float32 logit that a double's sigmoid does not follow: from
    about 24 on.  The sums 1 + exp(-x) lie on a grid of 2^-52, and exp(-x) is
    known to 2^-87: the reference's rounding is the kernel's."""
    E = 24
    g = gen(5)
    for base in (23.0, 24.0, 25.0, 30.0, 36.5):
        l = torch.full((5, E), base)
        for t in range(5):
            l[t] += 2.0 ** -19 * torch.randperm(E, generator=g).float()
        _, want = orc.route([l.double().numpy()], 7, score="sigmoid")
        with session(1):
            for bias in (None, torch.zeros(E, device=DEV)):
                _, e = rr.route([l.to(DEV)], 7, score="sigmoid", bias=bias)
                assert np.array_equal(e[0].cpu().numpy(), want[0]), f"at {base}, bias {bias is not None}"


# ---------------------------------------------------------------- groups masked by the lowest value

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [3.4028234663852886e38, 2.5e38])
def test_group_sums_past_float32(score, big):
    """A bias of the type's lowest value (or near its largest): two of them add
    up beyond float32, not beyond the 64 bits that decide."""
    E, G = 32, 4
    g = gen(3)
    l = torch.randn(20, E, generator=g)
    l[::2, :8] = -math.inf  # group 0 has nothing to choose
    low = torch.zeros(E)
    low[:24] = -big
    high = torch.zeros(E)
    high[8:16] = big * 0.9
    high[16:24] = big
    for bias in (low, high, -high):
        for top_groups in (1, 2, 3):
            K = 8 if top_groups == 1 else 12  # more than one group has
            kw = dict(score=score, groups=G, top_groups=top_groups, group_by="top2")
            _, want = orc.route([l.double().numpy()], K, bias=bias.double().numpy(), **kw)
            with session(1):
                for reps in (1, 120):
                    _, e = rr.route([l.repeat(reps, 1).to(DEV)], K, bias=bias.to(DEV), **kw)
                    got = e[0].cpu().numpy().reshape(reps, 20, K)
                    assert (got == want[0]).all(), f"bias {bias[0]}, {bias[8]}: {got[0]} not {want[0]}"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [3.4028234663852886e38, 2.5e38, -2.5e38])
def test_masked_experts_under_a_large_bias(score, big):
    """A margin beyond float32's range takes in no expert that is masked out."""
    E, K = 32, 6
    g = gen(4)
    l = torch.randn(20, E, generator=g)
    l[:, ::3] = -math.inf
    for bias in (torch.full((E,), big), torch.where(torch.arange(E) % 2 == 0, big, 0.0)):
        _, want = orc.route([l.double().numpy()], K, score=score, bias=bias.double().numpy())
        with session(1):
            for reps in (1, 120):
                _, e = rr.route([l.repeat(reps, 1).to(DEV)], K, score=score, bias=bias.to(DEV))
                got = e[0].cpu().numpy().reshape(reps, 20, K)
                assert (got == want[0]).all(), f"bias {bias[0]}, {bias[1]}: {got[0]} not {want[0]}"


# ---------------------------------------------------------------- a softmax over all experts

@pytest.mark.parametrize("E,K,bias", [(8, 2, False), (8, 6, False), (64, 4, False), (256, 8, False), (256, 8, True),
                                      (600, 12, False), (1000, 16, True)])
@pytest.mark.parametrize("std", [2, 6])
def test_weights_of_a_full_softmax(E, K, bias, std):
    """Rounded once, u, but for the sum's error: the terms of experts that were
    not chosen are float32 exponentials, each off by (2 t + 2) u at t below the
    largest logit (the roundings of t and of t log2 e, a step of v_exp)."""
    g = gen(E + K)
    l = torch.randn(2100, E, generator=g) * std
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    x = l.double()
    t = x.amax(1, keepdim=True) - x
    s = torch.exp(-t) / torch.exp(-t).sum(1, keepdim=True)
    for rows in (7, 2100):
        with session(1):
            w, e = rr.route([l[:rows].to(DEV)], K, bias=None if b is None else b.to(DEV), renormalize=False, scale=2.0)
        at = e[0].cpu().long()
        want = 2 * torch.gather(s[:rows], 1, at)
        other = (s * (2 * t + 2))[:rows].scatter(1, at, 0.0).sum(1, keepdim=True)
        off = (w[0].cpu().double() - want).abs() / want
        bound = U * (1 + other) * (1 + 2.0 ** -10)
        assert (off <= bound).all(), f"{rows} rows: {((off - bound) / U).max().item()} roundings past {other.max().item()}"


def exact_grad(x, experts, dw, renormalize):
    """d_logits of one token without cancellation: with D_e the sum of the
    d_weights of e's choices, d_e = s_e sum_j s_j (D_e - D_j); with renormalize
    the same over the choices, of weights q_k, added up for each expert.  With
    the sums of the added parts' sizes."""
    x = np.asarray(x, np.float64)
    if not renormalize:
        D = np.array([sum(d for e, d in zip(experts, dw) if e == j) for j in range(x.size)])
        s = np.exp(x - x.max())
        s /= math.fsum(s)
        out = np.array([s[e] * math.fsum(s * (D[e] - D)) for e in range(x.size)])
        return out, np.abs(out)
    dw = np.array(dw)
    q = np.exp(x[experts] - x[experts].max())
    q /= math.fsum(q)
    out, size = np.zeros_like(x), np.zeros_like(x)
    for e, p, d in zip(experts, q, dw):
        part = p * math.fsum(q * (d - dw))
        out[e] += part
        size[e] += abs(part)
    return out, size


@pytest.mark.parametrize("E", [8, 300])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_where_one_expert_outweighs_the_others(E, renormalize):
    """1 - p of a confident choice, against the exact gradient and relative to it:
    64-bit terms off by 2^-36 at most, added without cancellation, rounded to
    float32 once for a chosen expert; of the others six roundings, and their
    exponentials' arguments.  d_weights are whole numbers, so that their
    differences are exact."""
    gaps = [3, 9, 12, 15, 17, 20, 25, 40, 60]
    choose = [[5], [5, 2], [2, 5, 0], [2, 0], [5, 2, 5], [0, 2, 0]]
    for experts in choose:
        K = len(experts)
        l = torch.linspace(0.0, 1.0, E).repeat(len(gaps), 1)
        for t, gap in enumerate(gaps):
            l[t, 5] = float(gap) + 1
        dw = torch.tensor([[3.0, 3.0, -2.0][:K]] * len(gaps))
        ex = torch.tensor([experts] * len(gaps), dtype=torch.int32)
        with session(1):
            d = rr.route_grad([l.to(DEV)], [ex.to(DEV)], [dw.to(DEV)], renormalize=renormalize)[0].cpu().double().numpy()
        for t, gap in enumerate(gaps):
            x = l[t].double().numpy()
            want, size = exact_grad(x, experts, dw[t].tolist(), renormalize)
            bound = size * U * 1.001
            for e in set(experts):
                if renormalize and experts.count(e) > 1:  # each part is rounded, then their sum
                    bound[e] += np.abs(want[e]) * U * 1.001
            if not renormalize:
                for e in range(E):
                    if e not in experts:
                        bound[e] = np.abs(want[e]) * U * (8 + x.max() - x[e])
            over = np.abs(d[t] - want) - bound - 2.0 ** -149
            assert over.max() <= 0, f"{experts}, gap {gap}, expert {over.argmax()}: {d[t][over.argmax()]!r} not {want[over.argmax()]!r}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("E", [8, 300])
def test_gradient_of_masked_rows_is_zero(dtype, renormalize, E):
    """Rows masked out altogether whose experts are named all the same, and
    rows whose named experts alone are masked out."""
    l = torch.randn(6, E, generator=gen(1))
    l[0] = -math.inf
    l[1, [1, 3]] = -math.inf
    l[2] = -math.inf
    l[2, 5] = 1.0
    l[5] = -math.inf
    ex = torch.tensor([[1, 3]] * 5 + [[-1, 3]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 2.0]] * 6)
    with session(1):
        d = rr.route_grad([l.to(TYPES[dtype]).to(DEV)], [ex.to(DEV)], [dw.to(DEV)], renormalize=renormalize)[0].cpu()
    assert torch.isfinite(d).all()
    for t in (0, 1, 2, 5):
        assert not d[t].any(), f"row {t}: {d[t]}"
    assert d[3].any() and d[4].any()


# ---------------------------------------------------------------- what changes while a call reads its arguments

class Later:
    """A number whose reading does something first, as another thread might."""

    def __init__(self, value, act):
        self.value, self.act = value, act

    def __float__(self):
        self.act()
        return float(self.value)

    def __index__(self):
        self.act()
        return int(self.value)


@pytest.mark.parametrize("ranks", [1, 2, 4])
def test_a_session_opened_during_the_call_is_not_taken_for_the_first(ranks):
    def reopen():
        rr.reset()
        rr.register(ranks)

    ids = [torch.zeros(3, dtype=torch.int64, device=DEV) for _ in range(2)]
    tables = [torch.ones(5, 8, device=DEV) for _ in range(2)]
    dy = [torch.ones(3, 8, device=DEV) for _ in range(2)]
    experts = [torch.zeros(3, 1, dtype=torch.int32, device=DEV) for _ in range(2)]
    for call in (lambda: rr.embedding(ids, tables, scale=Later(1, reopen)),
                 lambda: rr.embedding_grad(ids, dy, 10, scale=Later(1, reopen)),
                 lambda: rr.route(dy, 2, scale=Later(1, reopen)),
                 lambda: rr.route_grad(dy, experts, [torch.ones(3, 1, device=DEV)] * 2, scale=Later(1, reopen)),
                 lambda: rr.dispatch_plan(experts, Later(4, reopen))):
        with session(2):
            with pytest.raises(rr.CollectiveError, match="closed") as e:
                call()
            assert e.value.code == rr.RC_ERR_INVALID_ARGUMENT


def test_an_allocation_that_fails_raises_torchs_error():
    """As torch's own functions do, so that a program can make its batch smaller;
    with this process held to a thousandth of the memory."""
    with session(1):
        ids, dy = [torch.zeros(4, dtype=torch.int32, device=DEV)], [torch.ones(4, 64, device=DEV)]
        want = rr.embedding_grad(ids, dy, 100)[0]
        torch.cuda.empty_cache()
        torch.cuda.set_per_process_memory_fraction(0.001)
        try:
            with pytest.raises(torch.OutOfMemoryError):
                rr.embedding_grad(ids, dy, 2**24)
        finally:
            torch.cuda.set_per_process_memory_fraction(1.0)
        assert torch.equal(rr.embedding_grad(ids, dy, 100)[0], want)
