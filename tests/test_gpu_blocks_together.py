"""Block operators as a program uses them together: a decoding step's block, a
training step, graphs, streams, threads, tensors past 2^31 elements.

Each chain is compared with its own steps in 64 bits (float32 products for the
experts on the CPU); the operators' bounds are tested by themselves elsewhere,
here a step's inputs are what the step before gave."""

import threading

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from gpu_util import session
from oracle import blocks as orc
from test_gpu_blocks import check_norm, norm_inputs, stored
from test_gpu_moe import check as check_moe
from test_gpu_moe import inputs as moe_inputs
from test_gpu_rows import DEV, TYPES, U, dev, f64, gen, near, normal

pytestmark = pytest.mark.gpu


def test_a_decoding_step():
    """embedding -> rms_norm to 8 bits -> route -> moe_layer -> rms_norm with the layer's output."""
    counts, V, D, E, K = [3, 0, 2, 4], 101, 256, 8, 2
    i = moe_inputs(counts, E, K, D, 96, "e4m3", "e4m3", 3)
    g = gen(1)
    ids = [torch.randint(0, V, (n,), generator=g) for n in counts]
    tables = [normal(g, v, D, dtype="bf16") for v in (26, 26, 26, 23)]
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16)] * 4
    gate = normal(g, E, D).to(DEV)
    with session(4):
        h = rr.embedding(dev(ids), dev(tables))
        codes, scales = rr.rms_norm(h, dev(w), quantize="e4m3")
        plain = rr.rms_norm(h, dev(w))
        weights, experts = rr.route([x.float() @ gate.t() for x in plain], K)
        gpu = {k: dev(i[k]) for k in ("gate_up", "down", "gate_up_scales", "down_scales")}
        y = rr.moe_layer(codes, weights, experts, scales=scales, **gpu)
        out, sums = rr.rms_norm(y, dev(w), residuals=h)
        torch.cuda.synchronize()
        cpu = lambda ts: [t.cpu() for t in ts]  # noqa: E731
        check_norm((codes, scales), cpu(h), None, w, "bf16", "e4m3", None)
        check_moe(y, dict(i, xs=cpu(codes), scales=cpu(scales), weights=cpu(weights), experts=cpu(experts)), "bf16")
        check_norm((out, sums), cpu(y), cpu(h), w, "bf16", None, None)


def test_a_training_step():
    """The norm's gradients synced over the ranks, clipped by their norm and stepped by; ranks stay alike."""
    R, D = 4, 300
    g = gen(2)
    x = [normal(g, 9 + r, D) for r in range(R)]
    w = (1 + 0.1 * torch.randn(D, generator=g))
    dy = [normal(g, 9 + r, D) for r in range(R)]
    with session(R):
        params = [{7: w.clone().to(DEV)} for _ in range(R)]
        state = rr.adamw_state(params)
        p, m, v = f64([w])[0], np.zeros(D), np.zeros(D)
        for t in (1, 2, 3):
            ws = [q[7] for q in params]
            before = f64([ws[0]])[0]
            _, dw = rr.rms_norm_grad(dev(dy), dev(x), ws)
            grads = rr.all_reduce_params([{7: d} for d in dw], "mean")
            norms = rr.grad_norm(grads)
            rr.adamw_step(state, grads, lr=0.1, norms=norms, max_norm=0.5)
            torch.cuda.synchronize()
            want = sum(orc.rms_norm_grad(f64(dy)[r], f64(x)[r], before, 1e-6)[1] for r in range(R)) / R
            size = sum(np.abs(f64(dy)[r]).sum(axis=0) for r in range(R)) / R
            near(f64([grads[0][7]])[0], want, 300 * U * 5 * size, "synced gradient")
            got = f64([grads[0][7]])[0]
            norm = np.sqrt((got ** 2).sum())
            assert norm > 0.5
            p, m, v = orc.adamw(before, got * (0.5 / norm), m, v, t, lr=0.1)
            near(f64([params[0][7]])[0], p, 100 * U * 0.2 + 4 * U * np.abs(p) + 1e-6, "stepped weight")
            for r in range(1, R):
                assert torch.equal(params[r][7], params[0][7])
            m, v = f64([state.m[0][7]])[0], f64([state.v[0][7]])[0]


def test_norms_in_a_graph():
    x, res, w = norm_inputs([5, 3], 1001, "bf16", "f32", 4)
    with session(2):
        xd, rd, wd = dev(x), dev(res), dev(w)
        out = rr.rms_norm(xd, wd, residuals=rd, quantize="e4m3", group=128)
        grads = rr.rms_norm_grad(rd, xd, wd)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rr.rms_norm(xd, wd, residuals=rd, quantize="e4m3", group=128, out=out)
            rr.rms_norm_grad(rd, xd, wd, out=grads)
        for k in range(4):
            for a in xd + rd + wd:
                a.mul_(-1.5 if k % 2 else 0.75)
            want = rr.rms_norm(xd, wd, residuals=rd, quantize="e4m3", group=128)
            want_g = rr.rms_norm_grad(rd, xd, wd)
            torch.cuda.synchronize()
            for lists in out + grads:
                for a in lists:
                    a.view(torch.uint8).zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out + grads, want + want_g):
                for p, q in zip(a, b):
                    assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_on_another_stream():
    x, res, w = norm_inputs([50, 70], 512, "bf16", "bf16", 6)
    i = moe_inputs([2, 3], 4, 2, 128, 64, "bf16", "bf16", 8)
    with session(2):
        xd, rd, wd = dev(x), dev(res), dev(w)
        gpu = {k: dev(t) if t is not None else None for k, t in i.items()}
        params = [{0: normal(gen(3), 5000).to(DEV)} for _ in range(2)]
        grads = [{0: normal(gen(4), 5000).to(DEV)} for _ in range(2)]
        state = rr.adamw_state(params)
        want = rr.rms_norm(xd, wd, residuals=rd)
        want_moe = rr.moe_layer(**gpu)
        want_norm = rr.grad_norm(grads)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        y, sums = rr.rms_norm(xd, wd, residuals=rd, stream=s)
        m = rr.moe_layer(**gpu, stream=s)
        n = rr.grad_norm(grads, stream=s)
        rr.adamw_step(state, grads, norms=n, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(y + sums + m + [n], want[0] + want[1] + want_moe + [want_norm]))
        assert state.step.tolist() == [1, 1]


def test_calls_from_two_threads():
    i = [moe_inputs([4, 4], 8, 2, 192, 64, "bf16", "bf16", 20 + k) for k in range(2)]
    with session(2):
        gpu = [{k: dev(t) if t is not None else None for k, t in x.items()} for x in i]
        want = [rr.moe_layer(**x) for x in gpu]
        torch.cuda.synchronize()
        bad = []

        def work(k):
            try:
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(50):
                        y = rr.moe_layer(**gpu[k])
                        n = rr.rms_norm(gpu[k]["xs"], [torch.ones(192, dtype=torch.bfloat16, device=DEV)] * 2)
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(y, want[k])) or not all(torch.isfinite(a).all() for a in n):
                        bad.append(k)
            except Exception as e:  # noqa: BLE001
                bad.append(repr(e))

        threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad


def test_tensors_past_2_31_elements():
    """The last rows, elements and experts of tensors whose offsets do not fit 32 bits."""
    with session(1):
        width = 32768
        rows = 2**31 // width + 3
        x = torch.zeros(rows, width, dtype=torch.bfloat16, device=DEV)
        g = gen(1)
        tail = normal(g, 3, width, dtype="bf16")
        x[-3:] = tail.to(DEV)
        w = [torch.ones(width, dtype=torch.bfloat16)]
        y = rr.rms_norm([x], dev(w))
        check_norm([y[0][-3:]], [tail], None, w, "bf16", None, None)
        assert not y[0][0].any()
        dx, dw = rr.rms_norm_grad([x], y, dev(w))
        want_x, _ = orc.rms_norm_grad(tail.double().numpy(), y[0][-3:].cpu().double().numpy(), np.ones(width), 1e-6)
        assert np.abs(dx[0][-3:].cpu().double().numpy() - want_x).max() < 2.0 ** -8 * np.abs(want_x).max() + 1e-3
        del x, y, dx
        torch.cuda.empty_cache()
        n = 2**31 + 1000
        p = torch.zeros(n, device=DEV)
        gr = torch.zeros(n, dtype=torch.float32, device=DEV)
        gr[-700:] = 3.0
        state = rr.adamw_state([{0: p}], bits=8)
        norms = rr.grad_norm([{0: gr}])
        rr.adamw_step(state, [{0: gr}], lr=0.5, weight_decay=0.0, norms=norms)
        torch.cuda.synchronize()
        near(norms.cpu().double().numpy(), [3 * 700 ** 0.5], 1e-5, "norm")
        assert torch.allclose(p[-700:], torch.full((700,), -0.5, device=DEV), rtol=1e-5) and not p[:-700].any()
        assert state.m[0][0][-700:].float().ne(0).all() and state.m_scale[0][0][-3:].ne(0).all()
        del p, gr, state
        torch.cuda.empty_cache()
        E, H, I = 72, 4096, 4096  # gate_up: 2.4e9 elements, the last expert's behind 2^31
        gu = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device=DEV)
        dn = torch.zeros(E, H, I, dtype=torch.bfloat16, device=DEV)
        gu[-1, :, 0] = 1.0
        dn[-1, -1, -1] = 2.0
        xs = torch.zeros(1, H, dtype=torch.bfloat16, device=DEV)
        xs[0, 0] = 1.0
        y = rr.moe_layer([xs], [torch.ones(1, 1, device=DEV)], [torch.full((1, 1), E - 1, dtype=torch.int32, device=DEV)], [gu], [dn])
        torch.cuda.synchronize()
        silu = 1 / (1 + np.exp(-1.0))
        assert abs(float(y[0][0, -1]) - 2 * silu) < 2.0 ** -7 and not y[0][0, :-1].any()


def test_nothing_to_do():
    """Ranks without tokens, parameters without elements or gradients."""
    with session(2):
        e = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
        w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
        y, s = rr.rms_norm([e, e], [w, w], residuals=[e, e])
        assert [t.shape for t in y + s] == [(0, 64)] * 4
        dx, dw = rr.rms_norm_grad([e, e], [e, e], [w, w])
        torch.cuda.synchronize()
        assert dx[0].shape == (0, 64) and not dw[0].any() and not dw[1].any()
        i = moe_inputs([0, 0], 4, 2, 64, 32, "bf16", "bf16", 1)
        y = rr.moe_layer(**{k: dev(t) if t is not None else None for k, t in i.items()})
        assert [t.shape for t in y] == [(0, 64)] * 2
        out = torch.ones(2, device=DEV)
        assert rr.grad_norm([{}, {}], out=out).tolist() == [0.0, 0.0]
        for bits in (32, 8):
            params = [{0: torch.zeros(0, device=DEV), 1: torch.ones(5, device=DEV)}, {}]
            state = rr.adamw_state(params, bits=bits)
            rr.adamw_step(state, [{0: torch.zeros(0, device=DEV)}, {}])
            rr.adamw_step(state, [{1: torch.ones(5, device=DEV)}, {}], lr=0.5, weight_decay=0.0, eps=0.0, betas=(0.0, 0.5))
            torch.cuda.synchronize()
            # counted at both calls: v = 0.5 of 1 - 0.5^2
            want = 1 - 0.5 / (0.5 / 0.75) ** 0.5
            assert state.step.tolist() == [2, 2] and torch.allclose(params[0][1], torch.full((5,), want, device=DEV), rtol=1e-6)


@pytest.mark.parametrize("where", ["the first call", "every call"])
def test_a_step_and_its_sync_in_one_graph(where):
    """grad_norm, adamw_step and a norm of the stepped weights captured together, replayed beside eager work."""
    with session(2):
        g = gen(11)
        make = lambda: [{0: torch.ones(512, device=DEV)} for _ in range(2)]  # noqa: E731
        eager, graphed = rr.adamw_state(make()), rr.adamw_state(make())
        grads = [{0: normal(g, 512).to(DEV)} for _ in range(2)]
        x = [normal(g, 7, 512).to(DEV) for _ in range(2)]
        norms = torch.zeros(2, device=DEV)
        out = [torch.zeros(7, 512, device=DEV) for _ in range(2)]

        def work(state, out):
            rr.grad_norm(grads, out=norms)
            rr.adamw_step(state, grads, lr=0.1, norms=norms, max_norm=1.0)
            rr.rms_norm(x, [m[0] for m in state.params], out=out)

        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            work(graphed, out)
        want = [torch.zeros(7, 512, device=DEV) for _ in range(2)]
        for k in range(3):
            if k == 0 or where == "every call":
                for m in grads:
                    m[0].mul_(-0.7)
            work(eager, want)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out + [m[0] for m in graphed.params], want + [m[0] for m in eager.params]):
                assert torch.equal(a, b)
