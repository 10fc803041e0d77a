"""The mixture-of-experts layer of a few tokens on the GPU against the oracle in
64 bits.

Error bound, with u = 2^-24: a sum of n products is off by at most (n / 4 + 16) * 2u
of its terms' sizes (each lane group sums a part; the matrix instructions'
sums are taken to be off by twice a float32 sum's), the exponential and the division by 4 u of
h and g's own by its size; hidden values as two bfloat16 numbers by 2^-16, and a
float16 weight's product without the two small parts by 2^-16: 3 * 2^-16 in all.
oracle.moe_token adds the sizes up.  The output adds half a step.
"""

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from gpu_util import session
from oracle import blocks as orc
from test_gpu_rows import DEV, HALF, TINY, TYPES, U, dev, f64, gen, near, normal, shifted

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def inputs(counts, experts, top_k, width, inner, dtype, weights, seed, padding=0.0):
    g = gen(seed)
    R, E = len(counts), experts
    eight = weights == "e4m3"
    def w(*shape):
        x = torch.randn(*shape, generator=g)
        return (x * 100).clamp(-448, 448).to(E4M3) if eight else (x * shape[-1] ** -0.5).to(TYPES[weights])
    if dtype == "e4m3":
        xs = [(torch.randn(n, width, generator=g) * 100).clamp(-448, 448).to(E4M3) for n in counts]
        scales = [0.005 + 0.01 * torch.rand(n, 1, generator=g) for n in counts]
    else:
        xs, scales = [normal(g, n, width, dtype=dtype) for n in counts], None
    gu, dn = [w(E // R, 2 * inner, width) for _ in range(R)], [w(E // R, width, inner) for _ in range(R)]
    gs = [(0.5 + torch.rand(E // R, 2 * inner, generator=g)) * 0.01 * width ** -0.5 for _ in range(R)] if eight else None
    ds = [(0.5 + torch.rand(E // R, width, generator=g)) * 0.01 * inner ** -0.5 for _ in range(R)] if eight else None
    ex, ws = [], []
    for n in counts:
        e = torch.argsort(torch.rand(n, E, generator=g), dim=1)[:, :top_k].to(torch.int32)
        gone = torch.rand(n, top_k, generator=g) < padding
        ex.append(torch.where(gone, -1, e).to(torch.int32).contiguous())
        ws.append(torch.rand(n, top_k, generator=g))
    return dict(xs=xs, weights=ws, experts=ex, gate_up=gu, down=dn, scales=scales, gate_up_scales=gs, down_scales=ds)


def on_gpu(i):
    return {k: dev(v) if v is not None else None for k, v in i.items()}


def check(ys, i, out):
    f = lambda ts: [t.float().double().numpy() for t in ts]  # noqa: E731
    xs, gu, dn = f(i["xs"]), np.concatenate(f(i["gate_up"])), np.concatenate(f(i["down"]))
    if i["scales"] is not None:
        xs = [x * s for x, s in zip(xs, f(i["scales"]))]
    if i["gate_up_scales"] is not None:
        gu = gu * np.concatenate(f(i["gate_up_scales"]))[..., None]
        dn = dn * np.concatenate(f(i["down_scales"]))[..., None]
    H, I, K = dn.shape[1], dn.shape[2], i["experts"][0].shape[1]
    wide = i["gate_up"][0].dtype == torch.float32
    rel = 1.01 * 2 * U * (H / 4 + I / 4 + 32 + K + 8) + (0 if wide else 3 * 2.0 ** -16)
    for r, x in enumerate(xs):
        for t in range(x.shape[0]):
            y, size = orc.moe_token(x[t], i["weights"][r][t].double().numpy(), i["experts"][r][t].numpy(), gu, dn)
            near(ys[r][t].float().cpu().double().numpy(), y, rel * size + HALF[out] * np.abs(y) * 1.01 + TINY[out], f"rank {r}, token {t}")


KINDS = [("f32", "f32", "f32"), ("f16", "f16", "f16"), ("bf16", "bf16", "bf16"), ("f16", "e4m3", "f16"), ("bf16", "e4m3", "bf16"),
         ("e4m3", "e4m3", "bf16"), ("e4m3", "e4m3", "f16"), ("e4m3", "e4m3", "f32")]
SHAPES = [
    # tokens of each rank, experts, top_k, width, inner
    ([1], 1, 1, 1, 1),
    ([1], 8, 2, 64, 64),
    ([1], 64, 8, 512, 192),
    ([3, 0, 2], 12, 4, 100, 37),
    ([5], 4, 3, 257, 130),
    ([17, 1], 6, 2, 333, 65),   # more than one tile of entries to an expert
    ([40], 3, 2, 96, 200),      # and more than two
    ([200], 2, 1, 130, 48),     # and more than four
    ([2, 2, 2, 2, 2, 2, 2, 2], 256, 8, 128, 64),
    ([64, 64], 16, 16, 48, 33),  # 2048 entries
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", KINDS, ids="-".join)
def test_layer(shape, kind):
    counts, experts, top_k, width, inner = shape
    i = inputs(counts, experts, top_k, width, inner, kind[0], kind[1], 7, padding=0.2 if sum(counts) > 4 else 0.0)
    with session(len(counts)):
        ys = rr.moe_layer(**on_gpu(i), dtype=TYPES[kind[2]])
        torch.cuda.synchronize()
        assert all(y.dtype == TYPES[kind[2]] for y in ys)
        check(ys, i, kind[2])


@pytest.mark.parametrize("kind", KINDS[:6], ids="-".join)
def test_rows_off_the_grid(kind):
    i = inputs([3, 4], 4, 2, 333, 65, kind[0], kind[1], 3)
    with session(2):
        g = on_gpu(i)
        for k in g:
            if g[k] is not None:
                g[k] = shifted(g[k], 3)
        ys = rr.moe_layer(**g, out=shifted([torch.zeros(n, 333, dtype=TYPES[kind[2]], device=DEV) for n in (3, 4)], 1))
        torch.cuda.synchronize()
        check(ys, i, kind[2])


def test_choices_that_repeat_or_name_none():
    """One expert twice in a token, experts out of range, tokens without any, their rows not numbers."""
    i = inputs([6], 4, 3, 128, 64, "bf16", "bf16", 5)
    i["experts"] = [torch.tensor([[1, 1, 2], [-1, -1, -1], [4, 0, -7], [2**31 - 1, 3, 3], [-1, 2, -1], [0, 1, 2]], dtype=torch.int32)]
    i["xs"][0][1] = float("nan")
    i["weights"][0][2, 0] = float("nan")  # of expert 4, that is none
    i["gate_up"][0][3, 5] = 0.0
    with session(1):
        ys = rr.moe_layer(**on_gpu(i))
        torch.cuda.synchronize()
    assert not ys[0][1].any()
    i["xs"][0][1] = 0
    i["weights"][0][2, 0] = 0
    check(ys, i, "bf16")


def test_a_row_that_is_not_finite_stays_alone():
    i = inputs([8], 2, 1, 256, 128, "bf16", "bf16", 9)
    i["experts"][0].zero_()
    with session(1):
        want = rr.moe_layer(**on_gpu(i))[0].clone()
        i["xs"][0][3, 10] = float("inf")
        i["xs"][0][5, 20] = float("nan")
        got = rr.moe_layer(**on_gpu(i))[0]
        torch.cuda.synchronize()
        for t in range(8):
            assert got[t].isnan().any() if t in (3, 5) else torch.equal(got[t], want[t]), t


def test_values_beyond_float16():
    """Hidden values past 65504, and far below its smallest, with float16 weights."""
    i = inputs([2], 2, 1, 64, 64, "f16", "f16", 11)
    i["experts"][0].copy_(torch.tensor([[0], [1]]))
    i["gate_up"][0][0] *= 200
    i["down"][0][0] *= 2.0 ** -12
    i["gate_up"][0][1] *= 2.0 ** -7
    with session(1):
        ys = rr.moe_layer(**on_gpu(i))
        torch.cuda.synchronize()
        check(ys, i, "f16")


@pytest.mark.parametrize("shape", [([60, 3], 4, 2, 130, 96), ([150], 2, 1, 200, 70), ([301], 2, 1, 65, 129), ([90, 90, 90], 3, 3, 1000, 67),
                                   ([700], 1, 1, 64, 64), ([40, 30], 32, 8, 129, 519), ([200], 16, 10, 70, 1030), ([300], 16, 1, 257, 1025),
                                   ([900, 100], 16, 2, 65, 1100), ([64], 64, 4, 64, 200)], ids=str)
@pytest.mark.parametrize("kind", KINDS, ids="-".join)
def test_experts_with_many_entries(shape, kind):
    """Tens and hundreds of entries to an expert: four and eight tiles of them, and more than one pass; with enough
    experts and rows for the way through LDS, and without."""
    counts, experts, top_k, width, inner = shape
    i = inputs(counts, experts, top_k, width, inner, kind[0], kind[1], 19, padding=0.1)
    if experts >= 16:  # popular experts, and some that nobody names
        for e in i["experts"]:
            e[:, 0] = torch.where(e[:, 0] >= 0, e[:, 0] % (experts // 8), -1)
    with session(len(counts)):
        ys = rr.moe_layer(**on_gpu(i), dtype=TYPES[kind[2]])
        torch.cuda.synchronize()
        check(ys, i, kind[2])


def test_a_token_among_others():
    """Bit for bit: what a token gives does not hang on which others there are, by either way of the sums."""
    for kind in (("bf16", "bf16"), ("e4m3", "e4m3")):
        for experts, n in ((8, 60), (64, 64)):
            i = inputs([n], experts, 8, 192, 260, *kind, 13)
            other = dict(i, xs=[i["xs"][0].flip(0)], experts=[i["experts"][0].clone()], weights=[i["weights"][0].flip(0)])
            other["experts"][0][:] = (other["experts"][0] + 1) % experts
            for k in ("xs", "weights", "experts"):
                other[k][0][11:14] = i[k][0][11:14]
            if i["scales"] is not None:
                other["scales"] = [i["scales"][0].flip(0)]
                other["scales"][0][11:14] = i["scales"][0][11:14]
            with session(1):
                a, b = rr.moe_layer(**on_gpu(i)), rr.moe_layer(**on_gpu(other))
                torch.cuda.synchronize()
                assert torch.equal(a[0][11:14], b[0][11:14]) and not torch.equal(a[0], b[0])


@pytest.mark.parametrize("kind", KINDS, ids="-".join)
@pytest.mark.parametrize("experts,width,inner", [(2, 192, 192), (2, 640, 448), (3, 645, 453), (2, 2048, 768), (16, 192, 1100)])
def test_a_token_in_a_growing_crowd(experts, width, inner, kind):
    """Bit for bit the same, whether its expert has one entry or several tiles of them, with the same sizes: the last
    shape through LDS, the others without."""
    n, token = 66, 5
    i = inputs([n], experts, 1, width, inner, *kind[:2], 23)
    with session(1):
        want = None
        for top in (1, 2, 16, 17, 32, 33, 48, 64, 65, 66):
            # expert 0's entries: this token and the last ones, so that its place among them changes too
            e = 1 + torch.arange(n, dtype=torch.int32) % (experts - 1)
            e[n - top:] = 0
            if n - top > token:
                e[n - top], e[token] = 1, 0
            assert int((e == 0).sum()) == top
            i["experts"] = [e.view(n, 1)]
            y = rr.moe_layer(**on_gpu(i), dtype=TYPES[kind[2]])[0]
            torch.cuda.synchronize()
            if want is None:
                want = y[token].clone()
                check([y], i, kind[2])
            assert torch.equal(y[token], want), top


def lone_products(n, experts, inner, dtype, weights, gate, up, down, seed):
    """Inputs of n tokens with one choice each, whose gates are large (silu(z) = z in float32 from 40 on) and whose rows
    have one element: the hidden value j of an entry is gate[e, j] * up[e, j] * x, and the output D times them."""
    x = torch.zeros(n, 64)
    x[:, 0] = 1.0
    gu = torch.zeros(experts, 2 * inner, 64)
    gu[:, :inner, 0], gu[:, inner:, 0] = gate, up
    t = dict(TYPES, e4m3=E4M3)
    g = gen(seed)
    return dict(xs=[x.to(t[dtype])], weights=[torch.ones(n, 1)], experts=[torch.randint(0, experts, (n, 1), generator=g, dtype=torch.int32)],
                gate_up=[gu.to(t[weights])], down=[down.to(t[weights])], scales=None, gate_up_scales=None, down_scales=None)


# entries of two experts without the way through LDS, and of 128 with it
CROWDS = [(1, 2), (30, 2), (60, 2), (200, 2), (512, 128), (1800, 128)]


@pytest.mark.parametrize("n,experts", CROWDS)
def test_float32_outputs_of_8bit_rows(n, experts):
    """Outputs that are the hidden values themselves, as of float32: g and u have two roundings each and their product
    one, the three numbers that hold it add up in the matrix instructions with two more of twice that: 9 u."""
    inner, g = 64, gen(29)
    code = torch.arange(1, inner + 1).float()  # 8-bit numbers up to 16, every one of four bits after
    down = torch.eye(inner).repeat(experts, 1, 1)
    i = lone_products(n, experts, inner, "e4m3", "e4m3", (code % 15 + 1)[None], (code % 13 - 6.5)[None], down, 31)
    i["scales"] = [1.0 + torch.rand(n, 1, generator=g)]
    i["gate_up_scales"] = [40.0 + 10 * torch.rand(experts, 2 * inner, generator=g)]
    i["down_scales"] = [torch.ones(experts, inner)]
    with session(1):
        y = rr.moe_layer(**on_gpu(i), dtype=torch.float32)[0]
        torch.cuda.synchronize()
    e = i["experts"][0][:, 0].long()
    w = i["gate_up"][0].double()[:, :, 0] * i["gate_up_scales"][0].double()
    gate, up = (w[e] * i["scales"][0].double()).split(inner, 1)
    want = gate * up
    assert gate.min() >= 40
    near(y.cpu().double().numpy(), want.numpy(), 9.1 * U * want.abs().numpy(), "hidden values")


@pytest.mark.parametrize("n,experts", CROWDS)
def test_float16_weights_less_their_first_eight_bits(n, experts):
    """Outputs (f + l) h - f h with f of eight bits and h of thirteen: l h, to which the smaller halves of the weight and
    of the hidden value add up to 2^-9 by themselves.  Sums of six terms up to f h, each off by 2 u at most, and half a
    step."""
    inner = 64
    j = torch.arange(inner // 2)
    weight = 1 + (37 * j % 1024).float() * 2.0 ** -10
    first = weight.to(torch.bfloat16).float()
    down = torch.zeros(experts, 64, inner)
    down[:, j, 2 * j], down[:, j, 2 * j + 1] = weight, -first
    up = (1 + ((torch.arange(experts)[:, None] * 91 + 53 * j + 5) % 1024).float() * 2.0 ** -10).repeat_interleave(2, 1)
    i = lone_products(n, experts, inner, "f16", "f16", torch.tensor(48.0), up, down, 33)
    with session(1):
        y = rr.moe_layer(**on_gpu(i))[0]
        torch.cuda.synchronize()
    e = i["experts"][0][:, 0].long()
    h = 48 * up.double()[e][:, ::2]
    want = torch.zeros(n, 64, dtype=torch.float64)
    want[:, :inner // 2] = (weight - first).double() * h
    bound = HALF["f16"] * want.abs() + TINY["f16"]
    bound[:, :inner // 2] += 12 * U * first.double() * h
    near(y.cpu().double().numpy(), want.numpy(), bound.numpy(), "small halves")


def test_graph_replays():
    i = inputs([2, 3], 8, 2, 256, 128, "bf16", "bf16", 15)
    with session(2):
        g = on_gpu(i)
        out = [torch.zeros(n, 256, dtype=torch.bfloat16, device=DEV) for n in (2, 3)]
        rr.moe_layer(**g, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rr.moe_layer(**g, out=out)
        for k in range(4):
            for x, e in zip(g["xs"], g["experts"]):
                x.mul_(-1.25)
                e.copy_((e + 1) % 8)
            want = rr.moe_layer(**g)
            torch.cuda.synchronize()
            for y in out:
                y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_against_dispatch_and_combine():
    """The layer is what dispatch, the experts' products and combine give, float32."""
    i = inputs([5, 9], 4, 2, 160, 96, "f32", "f32", 17, padding=0.1)
    with session(2):
        g = on_gpu(i)
        got = rr.moe_layer(**g)
        plan = rr.dispatch_plan(g["experts"], 4)
        rows = rr.dispatch(g["xs"], plan)
        results = []
        for d in range(2):
            y = torch.zeros_like(rows[d])
            at = plan.offsets[d].tolist()
            for e in range(2):
                x = rows[d][at[e]:at[e + 1]]
                a, b = (x @ g["gate_up"][d][e].t()).split(96, 1)
                y[at[e]:at[e + 1]] = (torch.nn.functional.silu(a) * b) @ g["down"][d][e].t()
            results.append(y)
        want = rr.combine(results, plan, g["weights"])
        for a, b in zip(got, want):
            assert torch.allclose(a, b, rtol=1e-4, atol=1e-5)
