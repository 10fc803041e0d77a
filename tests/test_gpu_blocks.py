"""Block operators on the GPU against the oracle in 64 bits: the norm.

Error bounds, with u = 2^-24 (float32) and h = eps / 2 of an output's type:
  - a sum of n float32 terms in any order is off by at most n u times the sum of
    their absolute values (first order; the factor 1.01 covers the rest).  A
    row's sums run over at most 64 elements in a lane, six steps over the lanes
    and 16 over the waves, with a product or two a term: 90 u;
  - a row's factor 1 / sqrt(mean + eps): half of 90 u, and four roundings: 50 u;
  - an output in type T adds h of its own value, in 8 bits half a step:
    2^-4 of the value, or half of the smallest code, 2^-10 of the scale.
The sums with the residual are compared bit for bit.
"""

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from gpu_util import session
from oracle import blocks as orc
from test_gpu_rows import DEV, HALF, TINY, TYPES, U, dev, f64, gen, near, normal, shifted

pytestmark = pytest.mark.gpu
EPS = 1e-6


def stored(x, res):
    """The sums with the residual as the operator stores them."""
    return [a if r is None else (a.float() + r.float()).to(a.dtype) for a, r in zip(x, res or [None] * len(x))]


def values(codes, scales, group):
    """What 8-bit rows stand for, in 64 bits."""
    c, s = codes.detach().cpu().float().double().numpy(), scales.detach().cpu().double().numpy()
    return c * np.repeat(s, group or c.shape[1], axis=1)[:, :c.shape[1]]


def norm_inputs(counts, width, dtype, weights, seed, residual=True):
    g = gen(seed)
    x = [normal(g, n, width, std=2.0, dtype=dtype) for n in counts]
    res = [normal(g, n, width, std=3.0, dtype=dtype) for n in counts] if residual else None
    w = [(1 + 0.3 * torch.randn(width, generator=g)).to(TYPES[weights]) for _ in counts]
    return x, res, w


def check_norm(got, x, res, w, dtype, quantize, group, eps=EPS):
    """got: rms_norm's answer for these inputs."""
    got = list(got) if quantize or res is not None else [got]
    ys = got.pop(0)
    scales = got.pop(0) if quantize else None
    s = stored(x, res)
    if res is not None:
        for r, (a, b) in enumerate(zip(got[0], s)):
            assert torch.equal(a.cpu(), b), f"sums of rank {r}"
    for r in range(len(x)):
        want, _ = orc.rms_norm(f64(s)[r], f64(w)[r], eps)
        if not want.size:
            assert ys[r].shape == want.shape
            continue
        rel = 1.01 * 54 * U
        if not quantize:
            near(f64(ys)[r], want, (rel + HALF[dtype]) * np.abs(want) + TINY[dtype], f"ys of rank {r}")
            continue
        most = orc.largest(want, group)
        near(f64(scales)[r], most / 448, (rel + 2 * U) * most / 448, f"scales of rank {r}")
        step = np.repeat(most / 448, group or want.shape[1], axis=1)[:, :want.shape[1]]
        bound = (2.0 ** -4 + 4 * rel) * np.abs(want) + (1 + 4 * rel) * 2.0 ** -10 * step
        near(values(ys[r], scales[r], group), want, bound, f"8-bit ys of rank {r}")


WIDTHS = [1, 3, 8, 31, 64, 100, 257, 512, 1001, 2048, 2050, 4096, 5003, 8192, 16384, 20001, 32768]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,weights", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_norm(width, dtype, weights):
    counts = [5, 0, 1]
    x, res, w = norm_inputs(counts, width, dtype, weights, width)
    xd, rd, wd = dev(x), dev(res), dev(w)
    with session(3):
        for quantize, group in ((None, None), ("e4m3", None), ("e4m3", 32), ("e4m3", 128), ("e4m3", 256)):
            for r in (rd, None):
                got = rr.rms_norm(xd, wd, eps=EPS, residuals=r, quantize=quantize, group=group)
                torch.cuda.synchronize()
                check_norm(got, x, res if r is not None else None, w, dtype, quantize, group)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("off", [1, 3])
def test_norm_of_rows_off_the_grid(dtype, off):
    x, res, w = norm_inputs([4, 3], 1001, dtype, "f32", off)
    with session(2):
        for quantize, group in ((None, None), ("e4m3", 64)):
            out = [torch.empty(n, 1001, dtype=torch.float8_e4m3fn if quantize else TYPES[dtype], device=DEV) for n in (4, 3)]
            lists = [[torch.empty(o.numel() + off, dtype=o.dtype, device=DEV)[off:].view(o.shape) for o in out]]
            if quantize:
                lists.append([torch.empty(n, 16, device=DEV) for n in (4, 3)])
            lists.append(shifted(dev(x), off))
            got = rr.rms_norm(shifted(dev(x), off), shifted(dev(w), off), eps=EPS, residuals=shifted(dev(res), off),
                              quantize=quantize, group=group, out=lists)
            torch.cuda.synchronize()
            check_norm(got, x, res, w, dtype, quantize, group)


@pytest.mark.parametrize("width", [64, 1001, 5000])
def test_norm_in_place(width):
    x, res, w = norm_inputs([3, 9], width, "bf16", "bf16", 3)
    with session(2):
        want = rr.rms_norm(dev(x), dev(w), residuals=dev(res))
        xd, rd = dev(x), dev(res)
        y, s = rr.rms_norm(xd, dev(w), residuals=rd, out=(xd, rd))
        assert y is xd and s is rd
        torch.cuda.synchronize()
        for a, b in zip(want[0] + want[1], y + s):
            assert torch.equal(a, b)


def test_norm_of_many_rows_is_that_of_each():
    """Bit for bit: a row's result does not hang on the others."""
    x, res, w = norm_inputs([3001], 257, "bf16", "f32", 8)
    with session(1):
        y, c, s = rr.rms_norm(dev(x), dev(w), residuals=dev(res), quantize="e4m3", group=32)
        for t in (0, 1, 2, 1500, 3000):
            a, b, d = rr.rms_norm([x[0][t:t + 1].to(DEV)], dev(w), residuals=[res[0][t:t + 1].to(DEV)], quantize="e4m3", group=32)
            assert torch.equal(a[0].view(torch.uint8), y[0][t:t + 1].view(torch.uint8))
            assert torch.equal(b[0], c[0][t:t + 1]) and torch.equal(d[0], s[0][t:t + 1])


def test_norm_at_the_edges_of_its_values():
    """Rows of zeros, tiny and huge rows, infinities and NaN, each beside an ordinary one."""
    g = gen(4)
    x = normal(g, 8, 300)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e-38
    x[4] *= 1e20  # squares of 1e40, beyond float32
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    w = torch.ones(300)
    with session(1):
        y = rr.rms_norm([x.to(DEV)], [w.to(DEV)], eps=EPS)[0].cpu()
        z = rr.rms_norm([x.to(DEV)], [w.to(DEV)], eps=0.0)[0].cpu()
        codes, scales = rr.rms_norm([x.to(DEV)], [w.to(DEV)], eps=EPS, quantize="e4m3")
        least = rr.rms_norm([x.to(DEV)], [w.to(DEV)], eps=1.0, quantize="e4m3")
        torch.cuda.synchronize()
    codes, scales = codes[0].cpu().float(), scales[0].cpu()
    want, _ = orc.rms_norm(x.double().numpy(), w.double().numpy(), EPS)
    for t in (0, 2, 3, 7):
        near(y[t].double().numpy(), want[t], 60 * U * np.abs(want[t]) + 2.0 ** -149, f"row {t}")
    assert not y[1].any() and not y[4].any() and not codes[1].any() and scales[1] == 0
    assert y[5].isnan()[7] and not y[5][:7].any() and not y[5][8:].any()
    assert y[6].isnan().all() and codes[6].isnan().all()
    assert z[1].isnan().all()  # 0 / 0 without eps
    # values below 2^-117 = 6e-36 have no 8-bit form (here 1e-38, 1e-35 before), larger ones one relative to their row
    assert not least[0][0].cpu().float()[3].any() and least[1][0][3] == 0 and least[0][0].cpu().float()[2].any()
    assert codes[3].any() and scales[3] > 0
    near(codes[2].double() * scales[2].double(), want[2], 2.0 ** -3.9 * np.abs(want[2]) + 2.0 ** -9.9 * np.abs(want[2]).max() / 448, "tiny row")


def grad_bound(dy, s, w, ds, eps, dtype, tokens):
    _, factor = orc.rms_norm(s, w, eps)
    n = s * factor
    inner = np.abs(dy * w * s).sum(axis=1, keepdims=True) * factor ** 2 / s.shape[1]
    # 50 u in each factor, 90 u in the inner product, a few roundings
    dx = 1.01 * U * (56 * np.abs(factor * dy * w) + 250 * np.abs(n) * inner)
    if ds is not None:
        dx = dx + U * np.abs(ds)
    return dx, 1.01 * U * (tokens + 24 + 56) * np.abs(dy * n).sum(axis=0)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,weights", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
def test_norm_grad(width, dtype, weights):
    counts = [7, 0, 1, 1100 if width < 300 else 37]
    s, _, w = norm_inputs(counts, width, dtype, weights, width + 1, residual=False)
    g = gen(width)
    dy = [normal(g, n, width, dtype=dtype) for n in counts]
    ds = [normal(g, n, width, dtype=dtype) for n in counts]
    with session(4):
        for more in (ds, None):
            dx, dw = rr.rms_norm_grad(dev(dy), dev(s), dev(w), eps=EPS, d_sums=dev(more) if more else None)
            torch.cuda.synchronize()
            for r in range(4):
                d = f64(more)[r] if more else None
                want_x, want_w = orc.rms_norm_grad(f64(dy)[r], f64(s)[r], f64(w)[r], EPS, d)
                bx, bw = grad_bound(f64(dy)[r], f64(s)[r], f64(w)[r], d, EPS, dtype, counts[r])
                near(f64(dx)[r], want_x, bx + HALF[dtype] * np.abs(want_x) * 1.001 + TINY[dtype], f"d_xs of rank {r}")
                near(f64(dw)[r], want_w, bw + HALF[weights] * np.abs(want_w) * 1.001 + TINY[weights], f"d_weights of rank {r}")


def test_norm_grad_in_place_and_again():
    s, _, w = norm_inputs([9, 4], 1001, "bf16", "bf16", 5, residual=False)
    g = gen(6)
    dy, ds = [[normal(g, n, 1001, dtype="bf16") for n in (9, 4)] for _ in range(2)]
    with session(2):
        want = rr.rms_norm_grad(dev(dy), dev(s), dev(w), d_sums=dev(ds))
        for which in (0, 1):
            a, b = dev(dy), dev(ds)
            out = rr.rms_norm_grad(a, dev(s), dev(w), d_sums=b, out=((a, b)[which], [torch.empty_like(x) for x in want[1]]))
            torch.cuda.synchronize()
            for p, q in zip(want[0] + want[1], out[0] + out[1]):
                assert torch.equal(p, q)
