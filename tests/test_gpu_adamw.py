"""Gradient norms and AdamW steps on the GPU against the oracle in 64 bits.

Error bounds, with u = 2^-24:
  - norms: squares and sums in 64 bits, rounded once: u, and 2^-40 for the sums;
  - m: three roundings of terms no larger than |b1 m| + |(1 - b1) g| and the
    constants' own: 4 u of that; g scaled: 2 u more.  v likewise, 8 u;
  - the update: m's error, v's halved by the root, and six roundings of factors:
    16 u of |b1 m| + |(1 - b1) g| times rate / denominator; p adds 3 u |p|;
  - 8-bit m: half a step, 2^-4 of the value or 2^-10 of the scale; the root of v:
    a whole step.
"""

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from gpu_util import session
from oracle import blocks as orc
from test_gpu_rows import DEV, HALF, TYPES, U, gen, near

pytestmark = pytest.mark.gpu
SIZES = [1, 3, 4, 255, 256, 257, 1000, 8191, 8192, 8193, 24577, 100001]


def d64(t):
    return t.detach().cpu().double().numpy().reshape(-1)


def make(sizes, ranks, dtype, grads, bits, seed, scale=1e-3):
    """(params, gradients, state) of maps with tensors of these sizes, after 7 steps' worth of means."""
    g = gen(seed)
    params = [{i: (torch.randn(n, generator=g) * 0.05).to(TYPES[dtype]).to(DEV) for i, n in enumerate(sizes)} for _ in range(ranks)]
    gs = [{i: (torch.randn(n, generator=g) * scale * torch.exp(torch.randn(n, generator=g))).to(TYPES[grads]).to(DEV)
           for i, n in enumerate(sizes)} for _ in range(ranks)]
    state = rr.adamw_state(params, bits=bits)
    for r in range(ranks):
        for i, n in enumerate(sizes):
            m = torch.randn(n, generator=g) * scale * 0.5
            v = (scale * (0.5 + torch.rand(n, generator=g))) ** 2
            if bits == 32:
                state.m[r][i].copy_(m)
                state.v[r][i].copy_(v)
                continue
            for name, x in (("m", m), ("v", v.sqrt())):
                b = torch.from_numpy(orc.blocks(x.numpy())).float()
                s = b.abs().amax(1) / 448
                c = (b / s[:, None]).clamp(-448, 448).view(-1)[:n].to(torch.float8_e4m3fn)
                getattr(state, name)[r][i].copy_(c)
                getattr(state, name + "_scale")[r][i].copy_(s)
    state.step += 7
    return params, gs, state


def read(state, r, i):
    """The state of one parameter in 64 bits: p, m, v (the mean of the squares)."""
    p = state.master[r][i] if i in (state.master or [{}] * 16)[r] else state.params[r][i]
    m, v = d64(state.m[r][i].float()), d64(state.v[r][i].float())
    if state.bits == 8:
        m = m * np.repeat(d64(state.m_scale[r][i]), 256)[:m.size]
        v = (v * np.repeat(d64(state.v_scale[r][i]), 256)[:v.size]) ** 2
    return d64(p), m, v


def check_step(state, r, i, before, grad, t, dtype, seed=0, lr=1e-3, wd=1e-2, betas=(0.9, 0.999), eps=1e-8):
    """The state after a step whose parts before were `before` (read), with the gradient in 64 bits as it is used."""
    p0, m0, v0 = before
    p, m, v = orc.adamw(p0, grad, m0, v0, t, lr, betas, eps, wd)
    am = np.abs(betas[0] * m0) + np.abs((1 - betas[0]) * grad)
    em, ev = 1.01 * 8 * U * am, 1.01 * 12 * U * v
    denom = np.sqrt(v / (1 - betas[1] ** t)) + eps
    ep = 1.01 * U * (24 * lr / (1 - betas[0] ** t) * am / denom + 4 * np.abs(p0)) + 1e-37
    what = f"rank {r}, parameter {i}: "
    got_p = state.master[r][i] if dtype != "f32" else state.params[r][i]
    near(d64(got_p), p, ep, what + "p")
    if dtype != "f32":
        assert torch.equal(state.params[r][i], got_p.to(TYPES[dtype])), what + "params"
    if state.bits == 32:
        near(d64(state.m[r][i]), m, em + 1e-44, what + "m")
        near(d64(state.v[r][i]), v, ev + 1e-44, what + "v")
        return
    for name, x, e in (("m", m, em), ("v", np.sqrt(v), 8 * U * np.sqrt(v))):
        most = np.abs(orc.blocks(x)).max(axis=1)
        s = d64(getattr(state, name + "_scale")[r][i])
        me = orc.blocks(e).max(axis=1) + 2 * U * most
        near(s, most / 448, me / 448 + 1e-44, what + name + " scale")
        code = d64(getattr(state, name)[r][i].float())
        unit = np.repeat(s, 256)[:x.size]
        if name == "m":
            near(code * unit, x, (2.0 ** -4 + 1e-5) * np.abs(x) + (2.0 ** -10 + 1e-6) * unit + np.repeat(me, 256)[:x.size], what + "8-bit m")
            continue
        # the root of v: the code below plus one step where the part above it and the chance reach one
        y = np.minimum(x / np.where(unit > 0, unit, 1), 448.0)
        step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
        c = orc.chances(x.size, t, seed)
        want = np.where(y > 0, np.maximum(np.minimum(np.floor(y / step + c) * step, 448.0), 2.0 ** -9), 0.0)
        part = y / step + c
        sure = np.abs(part - np.round(part)) > 1e-4  # the rest may fall either way, or lie at a border of the steps
        sure &= np.abs(y / 2.0 ** np.round(np.log2(np.maximum(y, 1e-9))) - 1) > 1e-5
        # without a gradient values stay on the codes, an eighth of them at borders
        assert sure.mean() > 0.8 or x.size < 100
        assert np.array_equal(code[sure], want[sure]), what + "8-bit root of v"
        near(code, y, step * 1.001 + 2.0 ** -9, what + "8-bit root of v")


CASES = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,grads", CASES)
def test_step(dtype, grads, bits):
    with session(2):
        params, gs, state = make(SIZES, 2, dtype, grads, bits, 1, scale=1e-2)
        state.step[1] += 5
        before = [[read(state, r, i) for i in range(len(SIZES))] for r in range(2)]
        rr.adamw_step(state, gs, seed=11)
        torch.cuda.synchronize()
        assert state.step.tolist() == [8, 13]
        for r in range(2):
            for i in range(len(SIZES)):
                check_step(state, r, i, before[r][i], d64(gs[r][i]), [8, 13][r], dtype, seed=11)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_zero(bits):
    """A new state, several steps, a gradient of zeros among them: bias corrections, empty blocks."""
    with session(1):
        g = gen(3)
        params = [{"a": torch.randn(700, generator=g).to(DEV), "b": torch.zeros(300, device=DEV)}]
        state = rr.adamw_state(params, bits=bits)
        for t in range(1, 6):
            gs = [{"a": (torch.randn(700, generator=g) * 0.1).to(DEV), "b": torch.zeros(300, device=DEV)}]
            if t == 3:
                gs[0]["a"].zero_()
            before = [read(state, 0, k) for k in "ab"]
            rr.adamw_step(state, gs, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.0)
            torch.cuda.synchronize()
            for b, k in zip(before, "ab"):
                check_step(state, 0, k, b, d64(gs[0][k]), t, "f32", lr=0.01, wd=0.0, betas=(0.8, 0.95), eps=1e-6)
        assert not params[0]["b"].any() and not read(state, 0, "b")[1].any() and not read(state, 0, "b")[2].any()


@pytest.mark.parametrize("dtype,grads", CASES)
def test_norms(dtype, grads):
    with session(3):
        _, gs, _ = make(SIZES + [70000], 3, dtype, grads, 32, 5, scale=0.1)
        gs[2] = {}
        gs[1][0] = None
        want = [np.sqrt(sum((d64(x) ** 2).sum() for x in m.values() if x is not None)) for m in gs]
        out = torch.empty(3, device=DEV)
        got = rr.grad_norm(gs, out=out)
        assert got is out
        near(d64(got), want, (U + 2.0 ** -40) * np.array(want), "norms")
        every = rr.grad_norm(gs, over="all")
        whole = np.sqrt((np.array(want) ** 2).sum())
        near(d64(every), [whole] * 3, (U + 2.0 ** -40) * whole, "norm of all")


def test_norms_of_many_tensors_and_large_values():
    with session(2):
        gs = [{i: torch.full((3,), 10.0 ** (i % 30 - 5), device=DEV) for i in range(401)}, {}]
        gs[1] = {i: torch.full((5,), 1e-30, device=DEV) for i in range(2)}
        want = [np.sqrt(sum(3 * float(gs[0][i][0]) ** 2 for i in gs[0])), np.sqrt(10) * float(gs[1][0][0])]
        got = d64(rr.grad_norm(gs))
        near(got, want, 1e-6 * np.array(want), "norms")
        gs[1][0][1] = float("nan")
        gs[0][7][2] = float("inf")
        got = rr.grad_norm(gs).tolist()
        assert got[0] == float("inf") and got[1] != got[1]


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_scaling_and_steps_left_out(bits):
    sizes = [300, 8193]
    with session(3):
        params, gs, state = make(sizes, 3, "bf16", "f32", bits, 9, scale=1.0)
        gs[1] = {i: x * 1e-3 for i, x in gs[1].items()}  # below the bound
        gs[2][1][77] = float("inf")
        norms = rr.grad_norm(gs)
        before = [[read(state, r, i) for i in range(2)] for r in range(3)]
        raw = [[x.clone() for x in (state.params[2][i], state.master[2][i], state.m[2][i].view(torch.uint8), state.v[2][i].view(torch.uint8))]
               for i in range(2)]
        rr.adamw_step(state, gs, norms=norms, max_norm=5.0, grad_scale=-0.5)
        torch.cuda.synchronize()
        assert state.step.tolist() == [8, 8, 7]
        n = d64(norms)
        assert 0.5 * n[0] > 5 > 0.5 * n[1]
        for r in range(2):
            factor = -0.5 * (5.0 / (0.5 * n[0]) if r == 0 else 1.0)
            for i in range(2):
                check_step(state, r, i, before[r][i], factor * d64(gs[r][i]), 8, "bf16")
        for i in range(2):
            now = (state.params[2][i], state.master[2][i], state.m[2][i].view(torch.uint8), state.v[2][i].view(torch.uint8))
            assert all(torch.equal(a, b) for a, b in zip(raw[i], now))


def states_equal(a, b):
    names = ["params", "m", "v"] + (["master"] if any(a.master) else []) + (["m_scale", "v_scale"] if a.bits == 8 else [])
    for name in names:
        for x, y in zip(getattr(a, name), getattr(b, name)):
            assert list(x) == list(y)
            for k in x:
                assert torch.equal(x[k].view(torch.uint8), y[k].view(torch.uint8)), (name, k)
    assert torch.equal(a.step, b.step)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_into_another_state(bits, dtype):
    """Bit for bit what the step in place gives, what it was before left alone; parameters without a gradient copied."""
    with session(2):
        _, gs, state = make(SIZES, 2, dtype, dtype, bits, 21)
        _, _, same = make(SIZES, 2, dtype, dtype, bits, 21)
        _, _, keep = make(SIZES, 2, dtype, dtype, bits, 21)
        _, _, out = make(SIZES, 2, dtype, dtype, bits, 22)
        del gs[0][3], gs[1][len(SIZES) - 1]
        gs[1][5] = None
        gs[1][6][0] = float("nan")
        norms = rr.grad_norm(gs)
        got = rr.adamw_step(state, gs, norms=norms, out=out, seed=3)
        assert got is out
        rr.adamw_step(same, gs, norms=norms, seed=3)
        torch.cuda.synchronize()
        states_equal(out, same)
        states_equal(state, keep)
        assert out.step.tolist() == [8, 7]


def test_many_small_tensors():
    """More parameters than one launch names; every rank's in another order."""
    with session(2):
        sizes = [1 + (37 * i) % 600 for i in range(1000)]
        g = gen(2)
        base = {i: torch.randn(n, generator=g) for i, n in enumerate(sizes)}
        grad = {i: torch.randn(n, generator=g) for i, n in enumerate(sizes)}
        order = list(base)[::-1]
        params = [{i: base[i].to(DEV) for i in base}, {i: base[i].to(DEV) for i in order}]
        gs = [{i: grad[i].to(DEV) for i in order}, {i: grad[i].to(DEV) for i in base}]
        states = rr.adamw_state(params, bits=8)
        for _ in range(3):
            rr.adamw_step(states, gs, seed=2)
        torch.cuda.synchronize()
        for i in base:  # ranks with the same parameters stay alike
            assert torch.equal(params[0][i], params[1][i])
            assert torch.equal(states.v[0][i].view(torch.uint8), states.v[1][i].view(torch.uint8))


def test_tensors_off_the_grid():
    """Parameters, gradients and 8-bit codes at odd elements of larger buffers."""
    with session(1):
        for dtype in ("f32", "bf16"):
            n = 9001
            g = gen(8)
            def at(x, off):
                big = torch.zeros(n + 8, dtype=x.dtype, device=DEV)
                big[off:off + n].copy_(x)
                return big, big[off:off + n]
            p = (torch.randn(n, generator=g)).to(TYPES[dtype])
            grad = torch.randn(n, generator=g).to(TYPES[dtype])
            plain = rr.adamw_state([{0: p.to(DEV)}], bits=8)
            bufs = [at(p, 3), at(p.float(), 1)] + [at(torch.zeros(n, dtype=torch.float8_e4m3fn), k) for k in (1, 3)]
            off = rr.AdamWState([{0: bufs[0][1]}], 8, [{0: bufs[2][1]}], [{0: bufs[3][1]}], torch.zeros(1, dtype=torch.int32, device=DEV),
                                master=[{0: bufs[1][1]}] if dtype != "f32" else None, m_scale=[{0: torch.zeros(36, device=DEV)}],
                                v_scale=[{0: torch.zeros(36, device=DEV)}])
            for _ in range(2):
                rr.adamw_step(plain, [{0: grad.to(DEV)}])
                rr.adamw_step(off, [{0: at(grad, 5)[1]}])
            torch.cuda.synchronize()
            states_equal(plain, off)
            for (big, _), o in zip(bufs, (3, 1, 1, 3)):
                raw = big.view(torch.uint8)
                es = big.element_size()
                if big is bufs[1][0] and dtype == "f32":
                    continue
                assert not raw[:o * es].any() and not raw[(o + n) * es:].any()


def test_rounding_by_chance_keeps_small_changes():
    """The root of v under gradients whose square is half of it: the exact mean after 400 steps, not the start."""
    with session(1):
        n = 256 * 64
        state = rr.adamw_state([{0: torch.zeros(n, device=DEV)}], bits=8)
        state.step += 10000
        g = torch.full((n,), 0.5 ** 0.5, device=DEV)
        g[::256] = 1.0  # holds the scale of each block
        state.v[0][0].copy_(torch.full((n,), 448.0).to(torch.float8_e4m3fn))
        state.v_scale[0][0].fill_(1 / 448)
        for _ in range(400):
            rr.adamw_step(state, [{0: g}], seed=4)
        torch.cuda.synchronize()
        root = state.v[0][0].float().cpu().double() * state.v_scale[0][0].cpu().double().repeat_interleave(256)
        v = (root ** 2).view(-1, 256)[:, 1:]
        # rounding the root by chance adds its variance to the mean of the squares: a step d is at most 2^-4 of the
        # value above and 2^-3 below, a rounding adds up to d^2 / 4, and after n steps no more than n * d^2 / 4 * 0.999^n;
        # but roundings are rare (the change is a fraction of the step): each step adds f (1 - f) d^2 with f d the
        # change of the root, 0.0005 * (1 - 0.5) of it at most, so below 0.00025 * d of the value each, 400 * 0.00025 / 16
        exact = 0.5 + 0.5 * 0.999 ** 400
        assert abs(v.mean().item() - exact) < 400 * 0.00025 / 16 * 2 + 0.01
        assert v.mean().item() < 0.9


def test_chances_are_even():
    c = orc.chances(1 << 18, 5, 1)
    assert abs(c.mean() - 0.5) < 5 * (1 / 12) ** 0.5 / 512
    assert np.histogram(c, 64)[0].std() < 2 * (1 << 9)
    assert abs(np.corrcoef(c[:-1], c[1:])[0, 1]) < 0.01 and abs(np.corrcoef(c, orc.chances(1 << 18, 6, 1))[0, 1]) < 0.01


@pytest.mark.parametrize("beta1", [0.9, 0.99])
def test_codes_of_means_without_a_gradient(beta1):
    """Every one of the smaller codes, with gradients of nothing, next to nothing, and more: by chance where the oracle
    says, to nearest otherwise; the parameter's step is that of any other element."""
    with session(1):
        n = 256 * 128
        j = torch.arange(n)
        code = (j % 120 + 1).to(torch.uint8).view(torch.float8_e4m3fn).float() * torch.where(j // 120 % 2 == 0, 1.0, -1.0)
        code[::256] = 448.0  # the block's scale
        scale = 2.0 ** -4
        g = torch.tensor([0.0, 2.0 ** -9, -2.0 ** -7, 2.0 ** -5, 40.0])[j // 240 % 5] * scale
        g[::256] = 448.0 * scale
        p = torch.randn(n, generator=gen(3)).to(DEV)
        state = rr.adamw_state([{0: p}], bits=8)
        state.step += 50
        state.m[0][0].copy_(code.to(torch.float8_e4m3fn))
        state.m_scale[0][0].fill_(scale)
        state.v[0][0].copy_(torch.full((n,), 64 * 2.0 ** -9).to(torch.float8_e4m3fn))
        state.v_scale[0][0].fill_(scale)
        before = read(state, 0, 0)
        rr.adamw_step(state, [{0: g.to(DEV)}], lr=0.01, betas=(beta1, 0.999), seed=77)
        torch.cuda.synchronize()
        want_p, m, v = orc.adamw(before[0], d64(g), before[1], before[2], 51, 0.01, (beta1, 0.999))
        y = m / (np.abs(orc.blocks(m)).max() / 448)
        chance = orc.chances(n, 51, 77, True)
        want, held = orc.mean_codes(y, d64(g), scale, beta1, chance)
        a, step = np.abs(y), orc.distance(np.abs(y))
        part = a / step % 1
        # the rest may fall either way: at a border of the chance or of the half, of the octaves, of the rule
        sure = np.where(held, np.abs((part + chance + 0.5) % 1 - 0.5) > 1e-4, np.abs(part - 0.5) > 1e-4)
        sure &= (np.abs((1 - beta1) * a / (step / 2) - 1) > 1e-5) & (np.abs(np.abs(np.log2(a)) % 1 - 0.5) < 0.4999)
        got = d64(state.m[0][0].float())
        assert sure.mean() > 0.8 and 0.02 < held.mean() < 0.7
        assert np.array_equal(got[sure], want[sure])
        assert (got != orc.e4m3(y))[held & sure].any()
        am = np.abs(beta1 * before[1]) + np.abs((1 - beta1) * d64(g))
        denom = np.sqrt(v / (1 - 0.999 ** 51)) + 1e-8
        near(d64(p), want_p, 1.01 * U * (24 * 0.01 / (1 - beta1 ** 51) * am / denom + 4 * np.abs(before[0])), "p")


def test_means_without_a_gradient_go():
    """As on the CPU: half of each block loses its gradient, one element holds its scale; from step 300 on the idle
    parameters have means of zero and do not move by a bit."""
    with session(1):
        n = 256 * 8
        g = gen(6)
        p = torch.zeros(n, device=DEV)
        state = rr.adamw_state([{0: p}], bits=8)
        idle = torch.arange(n, device=DEV) % 2 == 1
        noise = torch.randn(64, n, generator=g).to(DEV)
        noise[:, ::256] = 8.0
        quiet = torch.where(idle, 0.0, noise)
        for t in range(2000):
            rr.adamw_step(state, [{0: (noise if t < 20 else quiet)[t % 64]}], lr=0.01, weight_decay=0.0, seed=t)
            if t == 300:
                rest = p.clone()
        torch.cuda.synchronize()
        assert torch.equal(p[idle], rest[idle]) and p[idle].all() and not torch.equal(p, rest)
        assert not state.m[0][0].float()[idle].any()


def test_steps_captured_into_a_graph():
    """Replays go on counting; lr from the GPU; each replay bit for bit the eager step."""
    with session(2):
        _, gs, eager = make([1000, 257], 2, "bf16", "bf16", 8, 31, scale=0.5)
        _, _, graphed = make([1000, 257], 2, "bf16", "bf16", 8, 31, scale=0.5)
        lr = torch.full((1,), 1e-2, device=DEV)
        norms = torch.zeros(2, device=DEV)

        def step(state):
            rr.grad_norm(gs, out=norms)
            rr.adamw_step(state, gs, lr=lr, norms=norms, max_norm=1.0, seed=9)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=s):
                step(graphed)
        for k in range(4):
            lr.fill_(1e-2 / (k + 1))
            gs[0][0].mul_(1.5)
            if k == 2:
                gs[1][1][3] = float("inf")
            step(eager)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            states_equal(eager, graphed)
        assert eager.step.tolist() == [11, 9]


def awaiting_free():
    """Addresses of blocks that are freed, but wait for a stream."""
    return {b["address"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"] if b["state"] not in ("active_allocated", "inactive")}


@pytest.mark.parametrize("other", [False, True])
def test_state_dropped_under_a_step_on_another_stream(other):
    """What the step goes by stays until the stream is done with it, though the state that held it is gone."""
    sizes = [300, 8193, 70000]
    with session(2):
        _, gs, want = make(sizes, 2, "bf16", "bf16", 8, 41)
        rr.adamw_step(want, gs, seed=6)
        _, _, state = make(sizes, 2, "bf16", "bf16", 8, 41)
        _, _, out = make(sizes, 2, "bf16", "bf16", 8, 42)
        a = torch.randn(4096, 4096, device=DEV)
        keep = [getattr(x, k) for x in (state, out) for k in ("params", "m", "v", "step", "master", "m_scale", "v_scale")]
        got = out if other else state
        got = {k: getattr(got, k) for k in ("bits", "params", "m", "v", "step", "master", "m_scale", "v_scale")}
        torch.cuda.synchronize()
        before = awaiting_free()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            b = a
            for _ in range(60):
                b = a @ b * 1e-2
            rr.adamw_step(state, gs, seed=6, out=out if other else None)
        del state, out
        waiting = awaiting_free() - before
        done = s.query()  # if the stream had been done by then, nothing would have to wait
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in range(512, 1 << 16, 512)]
        s.synchronize()
        assert done or len(waiting) == (2 if other else 1)
        torch.empty(1, device=DEV)  # takes note of what is done
        assert not waiting & awaiting_free()
        del junk, keep
        states_equal(rr.AdamWState(**got), want)


def test_a_step_on_a_stream_of_the_callers():
    """A stream that torch does not know is not asked for once the step is done: it may be gone."""
    with session(1):
        _, gs, want = make([5000], 1, "f32", "f32", 32, 43)
        rr.adamw_step(want, gs)
        _, _, state = make([5000], 1, "f32", "f32", 32, 43)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        before = awaiting_free()
        rr.adamw_step(state, gs, stream=s.cuda_stream)
        s.synchronize()
        states_equal(state, want)
        keep = state.params, state.m, state.v
        del state
        assert awaiting_free() <= before and keep


def test_state_whose_tensors_moved_is_refused():
    with session(1):
        p = torch.randn(100, device=DEV)
        state = rr.adamw_state([{0: p}])
        p.data = torch.randn(100, device=DEV)
        with pytest.raises(rr.CollectiveError, match="other memory"):
            rr.adamw_step(state, [{0: torch.randn(100, device=DEV)}])


def test_gradients_that_do_not_fit_are_refused():
    """Another shape, type, device or layout, and gradients of parameters that are not there: nothing is changed."""
    with session(1):
        p = torch.randn(4, 6, device=DEV)
        state = rr.adamw_state([{0: p, 1: torch.ones(3, device=DEV).half()}])
        keep = p.clone()
        good = torch.randn(4, 6, device=DEV)
        for grads in ([{0: good.t().contiguous()}], [{0: good.view(-1)}], [{0: good[:2]}], [{0: good.t().contiguous().t()}], [{0: good.bfloat16()}],
                      [{0: good.double()}], [{0: good.cpu()}], [{2: good}], [{0: 1.0}], [good], [], [{0: p}], [{1: torch.ones(3, device=DEV).bfloat16()}]):
            with pytest.raises((rr.CollectiveError, TypeError)):
                rr.adamw_step(state, grads)
        for kw in (dict(lr=-1.0), dict(lr=torch.ones(2, device=DEV)), dict(lr=torch.ones(1)), dict(lr=torch.ones(1, device=DEV).double()),
                   dict(norms=torch.ones(2, device=DEV)), dict(max_norm=1.0), dict(seed=-1), dict(seed=2**32), dict(betas=(0.9, 1.0)),
                   dict(out=rr.adamw_state([{0: torch.zeros(4, 6, device=DEV)}])), dict(out=rr.adamw_state([{0: p, 1: torch.ones(3, device=DEV).half()}])),
                   dict(out=rr.adamw_state([{0: torch.zeros(4, 6, device=DEV), 1: torch.ones(3, device=DEV).half()}], bits=8))):
            with pytest.raises((rr.CollectiveError, TypeError)):
                rr.adamw_step(state, [{0: good}], **kw)
        torch.cuda.synchronize()
        assert torch.equal(p, keep) and state.step.tolist() == [0]
        rr.adamw_step(state, [{0: good}])
        assert not torch.equal(p, keep)
    with session(2):
        with pytest.raises(rr.CollectiveError, match="ranks"):
            rr.adamw_step(state, [{}, {}])
