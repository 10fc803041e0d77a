"""Row exchanges on the CPU: the oracle against brute force and differences,
and every refusal of the C ABI (validate_only sessions, fake addresses) and of
the binding (host tensors)."""

import ctypes

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from oracle import rows as orc
from rank_reductions_amd import rows

OK, NR, INVAL = rr.RC_OK, rr.RC_ERR_NOT_REGISTERED, rr.RC_ERR_INVALID_ARGUMENT
SHAPE, DTYPE = rr.RC_ERR_SHAPE_MISMATCH, rr.RC_ERR_DTYPE_MISMATCH
R = 4
MiB = 1 << 20


# ---------------------------------------------------------------- the oracle

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("top_k", [1, 3])
def test_route_gradient_against_differences(score, renormalize, top_k):
    rng = np.random.default_rng(5)
    x = rng.normal(size=9)
    kw = dict(score=score, renormalize=renormalize, scale=1.75)
    w, e = orc.route_token(x, top_k, **kw)
    dw = rng.normal(size=top_k)
    got = orc.route_grad_token(x, e, dw, **kw)
    h = 1e-6
    for j in range(9):
        step = np.zeros(9)
        step[j] = h

        def weighted(y):
            s = orc._scores(y, score)[e]
            s = s / s.sum() if renormalize else s
            return (1.75 * s * dw).sum()

        want = (weighted(x + step) - weighted(x - step)) / (2 * h)
        assert abs(got[j] - want) < 1e-8


def test_route_token_by_hand():
    w, e = orc.route_token([1.0, 3.0, 3.0, -np.inf], 4)
    assert e.tolist() == [1, 2, 0, -1] and w[3] == 0 and abs(w.sum() - 1) < 1e-15
    w, e = orc.route_token([-np.inf] * 4, 2)
    assert e.tolist() == [-1, -1] and not w.any()
    # the best expert's group loses to the group whose two best add up to more
    _, e = orc.route_token([2.0, -9.0, 1.0, 1.0], 2, score="sigmoid", groups=2, top_groups=1, group_by="top2")
    assert e.tolist() == [2, 3]
    _, e = orc.route_token([2.0, -9.0, 1.0, 1.0], 2, score="sigmoid", groups=2, top_groups=1, group_by="max")
    assert e.tolist() == [0, 1]
    # a bias moves the choice, not the weight
    w, e = orc.route_token([0.0, 0.0], 1, score="sigmoid", bias=[0.0, 0.1], renormalize=False)
    assert e.tolist() == [1] and w[0] == 0.5


def test_plan_by_hand():
    ex = [np.array([[0, 3], [1, -1]], np.int32), np.array([[3, 0]], np.int32)]
    slots, offsets, counts = orc.dispatch_plan(ex, 4, [2, 9])
    assert slots[0].tolist() == [[0, 0], [-1, -1]] and slots[1].tolist() == [[1, 1]]
    assert [o.tolist() for o in offsets] == [[0, 2, 2], [0, 0, 2]]
    assert [c.tolist() for c in counts] == [[2, 1], [0, 2]]


def test_embedding_grad_orders_agree():
    rng = np.random.default_rng(7)
    ids = [rng.integers(-1, 4, size=n) for n in (300, 0, 41)]
    d = [rng.normal(size=(i.size, 3)) for i in ids]
    exact, size, count = orc.embedding_grad(ids, d, 3, 0.5)
    near = orc.embedding_grad_ordered(ids, d, 3, 0.5)
    assert np.all(np.abs(near - exact) <= 2.0 ** -24 * 80 * size + 1e-30)
    assert count.max() > orc.PIECE  # one id longer than a piece


# ---------------------------------------------------------------- the C ABI

@pytest.fixture
def lib():
    lib = rr.library()
    lib.rc_reset()
    cfg = rr.make_config(validate_only=True)
    assert lib.rc_register(R, ctypes.byref(cfg)) == OK
    yield lib
    lib.rc_reset()


class Space:
    """Fake addresses that do not overlap."""

    def __init__(self):
        self.at = 1 << 32

    def take(self, bytes_):
        p = self.at
        self.at += (bytes_ + MiB) // MiB * MiB
        return p


def ptrs(values):
    return (ctypes.c_void_p * len(values))(*values)


def route_call(grad=False, **kw):
    """(arguments of rc_route or rc_route_grad, everything that they point to)."""
    o = dict(dtype=rr.RC_F32, E=16, K=4, score=0, groups=1, top_groups=1, group_by=0, scale=1.0, size=None,
             tokens=[5, 0, 7, 1], logits=None, second=None, third=None, fourth=None, bias=None)
    o.update(kw)
    sp = Space()
    d = rows.RcRouteDesc(o["size"] if o["size"] is not None else ctypes.sizeof(rows.RcRouteDesc), o["dtype"], o["E"],
                         o["K"], o["score"], o["groups"], o["top_groups"], o["group_by"], 1, o["scale"], o["bias"])
    tokens = (ctypes.c_int64 * R)(*o["tokens"])
    arrays = [ptrs(o[n] or [sp.take(4096) for _ in range(R)]) for n in ("logits", "second", "third")]
    if grad:
        arrays.append(ptrs(o["fourth"] or [sp.take(4096) for _ in range(R)]))
    return [ctypes.byref(d), tokens, *arrays, None], (d, tokens, arrays)


@pytest.mark.parametrize("bad", [
    dict(size=8), dict(dtype=rr.RC_I32), dict(dtype=9), dict(E=0), dict(E=1025), dict(K=0), dict(K=17, E=64),
    dict(K=17), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=65, E=65 * 2),
    dict(groups=4, top_groups=5), dict(groups=4, top_groups=0), dict(group_by=2), dict(groups=8, top_groups=1, K=3),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=[1, -1, 0, 0]), dict(tokens=[2**31, 0, 0, 0]),
    dict(tokens=[2**30, 2**30, 2**30, 0]), dict(bias=1 << 40 | 2),
    dict(logits=[0, 1 << 40, 2 << 40, 3 << 40]),                         # NULL with tokens
    dict(logits=[(1 << 40) + 2, 2 << 40, 3 << 40, 4 << 40]),             # off the element size
    dict(second=[1 << 40, 2 << 40, 1 << 40, 3 << 40]),                   # two outputs in one place
    dict(second=[1 << 40, 2 << 40, 3 << 40, 4 << 40], third=[(1 << 40) + 16, 5 << 40, 6 << 40, 7 << 40]),
    dict(logits=[1 << 40, 2 << 40, 3 << 40, 4 << 40], second=[(1 << 40) + 4 * 5 * 16 - 4, 5 << 40, 6 << 40, 7 << 40]),
])
@pytest.mark.parametrize("grad", [False, True])
def test_route_refusals(lib, bad, grad):
    if grad and "second" in bad:
        bad = {("fourth" if k == "second" else "second" if k == "third" else k): v for k, v in bad.items()}
    args, keep = route_call(grad, **bad)
    fn = lib.rc_route_grad if grad else lib.rc_route
    assert fn(*args) == INVAL and lib.rc_last_error()


def test_route_accepts(lib):
    for kw in (dict(), dict(dtype=rows.RC_BF16), dict(E=1024, K=16), dict(E=64, groups=64, top_groups=16, K=16),
               dict(tokens=[0, 0, 0, 0], logits=[None] * R, second=[None] * R, third=[None] * R),
               dict(logits=[1 << 40, None, 3 << 40, 4 << 40]), dict(bias=1 << 40)):
        args, keep = route_call(**kw)
        assert lib.rc_route(*args) == OK, lib.rc_last_error()
        if kw.get("tokens") != [0] * R:
            args, keep = route_call(True, **kw)
            assert lib.rc_route_grad(*args) == OK, lib.rc_last_error()
    for i in range(5):  # NULL arguments
        args, keep = route_call()
        args[i] = None
        assert lib.rc_route(*args) == INVAL


def exchange_desc(**kw):
    o = dict(dtype=rr.RC_F32, E=16, K=2, width=32, tokens=[5, 0, 7, 1], capacity=[9, 0, 8, 26], size=None,
             experts=None, slots=None)
    o.update(kw)
    sp = Space()
    d = rows.RcExchangeDesc(o["size"] if o["size"] is not None else ctypes.sizeof(rows.RcExchangeDesc), o["dtype"],
                            o["E"], o["K"], o["width"])
    held = [(ctypes.c_int64 * R)(*o["tokens"]), (ctypes.c_int64 * R)(*o["capacity"]),
            ptrs(o["experts"] or [sp.take(4096) for _ in range(R)]),
            ptrs(o["slots"] or [sp.take(4096) for _ in range(R)])]
    d.tokens, d.capacity, d.experts, d.slots = map(ctypes.addressof, held)
    d.held = held
    return d, sp


def exchange_calls(lib, **kw):
    """Every exchange entry point on the same descriptor, as {name: status}."""
    own = {k: kw.pop(k) for k in list(kw) if k.startswith("buf")}
    d, sp = exchange_desc(**kw)
    ref = ctypes.byref(d)
    size = ctypes.c_int64(-1)
    b = [ptrs(own.get(f"buf{i}") or [sp.take(8192) for _ in range(R)]) for i in range(5)]
    got = {"plan_workspace": lib.rc_dispatch_plan_workspace(ref, ctypes.byref(size))}
    got["plan"] = lib.rc_dispatch_plan(ref, b[0], b[1], sp.take(1 << 20), 1 << 20, None)
    got["dispatch"] = lib.rc_dispatch(ref, b[0], b[1], None)
    got["combine"] = lib.rc_combine(ref, b[0], b[1], b[2], None)
    got["combine_plain"] = lib.rc_combine(ref, b[0], None, b[2], None)
    got["combine_grad"] = lib.rc_combine_grad(ref, b[0], b[1], b[2], b[3], b[4], None)
    return got


def test_exchange_accepts(lib):
    for kw in (dict(), dict(dtype=rows.RC_F16), dict(K=16), dict(width=1), dict(tokens=[0] * R), dict(capacity=[0] * R)):
        assert set(exchange_calls(lib, **kw).values()) == {OK}, (kw, lib.rc_last_error())


@pytest.mark.parametrize("bad", [dict(size=4), dict(E=0), dict(E=18), dict(E=1028), dict(K=0), dict(K=17),
                                 dict(tokens=[1, 2, 3, -4]), dict(tokens=[2**30, 0, 0, 0]), dict(capacity=[1, 2, 3, -1]),
                                 dict(capacity=[2**31, 0, 0, 0])])
def test_exchange_refusals(lib, bad):
    assert set(exchange_calls(lib, **bad).values()) == {INVAL}


@pytest.mark.parametrize("bad", [dict(dtype=rr.RC_I32), dict(dtype=rows.RC_I64), dict(width=0), dict(width=2**22 + 1)])
def test_exchange_refuses_rows(lib, bad):
    got = exchange_calls(lib, **bad)
    assert got.pop("plan") == OK and got.pop("plan_workspace") == OK
    assert set(got.values()) == {INVAL}


def test_exchange_buffers(lib):
    far = [(i + 1) << 40 for i in range(R)]
    got = exchange_calls(lib, experts=[None] + far[1:])
    assert got.pop("plan_workspace") == OK and set(got.values()) == {INVAL}
    got = exchange_calls(lib, slots=[far[0] + 2] + far[1:])
    assert got.pop("plan_workspace") == OK and set(got.values()) == {INVAL}
    # outputs over the plan's slots, over inputs, over one another
    for i, names in ((0, ["plan"]), (1, ["plan", "dispatch"]), (2, ["combine", "combine_plain"]),
                     (3, ["combine_grad"]), (4, ["combine_grad"])):
        got = exchange_calls(lib, slots=far, **{f"buf{i}": [far[2]] + [(i + 9) << 40 for i in range(3)]})
        for n in names:
            assert got[n] == INVAL, (i, n)
    got = exchange_calls(lib, buf0=far, buf1=far)
    assert got["dispatch"] == INVAL and got["plan"] == INVAL and got["combine"] == OK
    got = exchange_calls(lib, buf1=far, buf3=far)
    assert got["combine_grad"] == INVAL  # d_rows over rows
    # NULL arrays
    d, sp = exchange_desc()
    b = ptrs([sp.take(4096) for _ in range(R)])
    assert lib.rc_dispatch(ctypes.byref(d), None, b, None) == INVAL
    assert lib.rc_dispatch(None, b, b, None) == INVAL
    d.slots = None
    assert lib.rc_dispatch(ctypes.byref(d), b, b, None) == INVAL


def test_plan_workspace_is_checked(lib):
    d, sp = exchange_desc(tokens=[20000, 3, 0, 20000], K=4, E=64,
                          experts=[(i + 1) << 40 for i in range(R)], slots=[(i + 11) << 40 for i in range(R)])
    size = ctypes.c_int64()
    assert lib.rc_dispatch_plan_workspace(ctypes.byref(d), ctypes.byref(size)) == OK and size.value > 0
    out = [ptrs([sp.take(4096) for _ in range(R)]) for _ in range(2)]
    at = sp.take(size.value)
    assert lib.rc_dispatch_plan(ctypes.byref(d), *out, at, size.value, None) == OK
    assert lib.rc_dispatch_plan(ctypes.byref(d), *out, at, size.value - 1, None) == INVAL
    assert lib.rc_dispatch_plan(ctypes.byref(d), *out, None, size.value, None) == INVAL
    assert lib.rc_dispatch_plan(ctypes.byref(d), *out, at + 4, size.value, None) == INVAL
    assert lib.rc_dispatch_plan(ctypes.byref(d), *out, 1 << 40, size.value, None) == INVAL  # over the experts


def embedding_calls(lib, **kw):
    o = dict(dtype=rr.RC_F32, id=rr.RC_I32, grad=rr.RC_F32, acc=0, scale=1.0, vocab=10, width=32, tokens=[5, 0, 7, 1],
             size=None, ids=None, buf0=None, buf1=None, workspace=None, workspace_bytes=None)
    o.update(kw)
    sp = Space()
    d = rows.RcEmbeddingDesc(o["size"] if o["size"] is not None else ctypes.sizeof(rows.RcEmbeddingDesc), o["dtype"],
                             o["id"], o["grad"], o["acc"], o["scale"], o["vocab"], o["width"])
    held = [(ctypes.c_int64 * R)(*o["tokens"]), ptrs(o["ids"] or [sp.take(4096) for _ in range(R)])]
    d.tokens, d.ids = map(ctypes.addressof, held)
    b = [ptrs(o[f"buf{i}"] or [sp.take(8192) for _ in range(R)]) for i in range(2)]
    size = ctypes.c_int64()
    ref = ctypes.byref(d)
    got = {"lookup": lib.rc_embedding(ref, b[0], b[1], None),
           "workspace": lib.rc_embedding_grad_workspace(ref, ctypes.byref(size))}
    n = o["workspace_bytes"] if o["workspace_bytes"] is not None else size.value
    got["grad"] = lib.rc_embedding_grad(ref, b[0], b[1], o["workspace"] or sp.take(max(n, 1)), n, None)
    return got


def test_embedding_accepts(lib):
    for kw in (dict(), dict(dtype=rows.RC_BF16, grad=rows.RC_BF16), dict(dtype=rows.RC_F16, id=rows.RC_I64),
               dict(tokens=[0] * R), dict(vocab=1, buf0=[1 << 40, 2 << 40, 3 << 40, 4 << 40]), dict(vocab=2), dict(width=1)):
        assert set(embedding_calls(lib, **kw).values()) == {OK}, (kw, lib.rc_last_error())
    # a vocabulary of 5 over 4 ranks: segments of 2, 2, 1 and 0 rows
    assert embedding_calls(lib, vocab=5, buf0=[1 << 40, 2 << 40, 3 << 40, None])["lookup"] == OK
    assert embedding_calls(lib, vocab=5, buf0=[1 << 40, 2 << 40, None, None])["lookup"] == INVAL


@pytest.mark.parametrize("bad", [dict(size=1), dict(dtype=rr.RC_I32), dict(id=rr.RC_F32), dict(vocab=0),
                                 dict(vocab=2**31 - 1), dict(width=0), dict(width=2**22 + 1), dict(scale=float("nan")),
                                 dict(tokens=[-1, 0, 0, 0]), dict(tokens=[2**31, 0, 0, 0])])
def test_embedding_refusals(lib, bad):
    assert set(embedding_calls(lib, **bad).values()) == {INVAL}


def test_embedding_buffers(lib):
    far = [(i + 1) << 40 for i in range(R)]
    got = embedding_calls(lib, dtype=rows.RC_F16, grad=rows.RC_BF16)
    assert got["lookup"] == OK and got["grad"] == INVAL and got["workspace"] == INVAL
    got = embedding_calls(lib, ids=[None] + far[1:])
    assert got["lookup"] == INVAL and got["grad"] == INVAL
    got = embedding_calls(lib, id=rows.RC_I64, ids=[far[0] + 4] + far[1:])
    assert got["lookup"] == INVAL and got["grad"] == INVAL
    got = embedding_calls(lib, buf0=far, buf1=far)
    assert got["lookup"] == INVAL and got["grad"] == INVAL
    got = embedding_calls(lib, ids=[far[0]] * R)  # one list of ids for all ranks
    assert got["lookup"] == OK and got["grad"] == OK
    assert embedding_calls(lib, workspace_bytes=0)["grad"] == INVAL
    assert embedding_calls(lib, workspace=(1 << 40) + 8)["grad"] == INVAL
    assert embedding_calls(lib, buf1=far, workspace=far[0])["grad"] == INVAL


def test_needs_a_whole_call_session():
    lib = rr.library()
    lib.rc_reset()
    args, keep = route_call()
    assert lib.rc_route(*args) == NR
    n = ctypes.c_int()
    assert lib.rc_session_info(ctypes.byref(n), None) == NR
    assert set(exchange_calls(lib).values()) == {NR} and set(embedding_calls(lib).values()) == {NR}
    cfg = rr.make_config(validate_only=True)
    assert lib.rc_rank_register(0, 1, ctypes.byref(cfg)) == OK
    assert lib.rc_route(*args) == INVAL and set(exchange_calls(lib).values()) == {INVAL}
    lib.rc_reset()


def test_session_info(lib):
    n, d = ctypes.c_int(), ctypes.c_int(7)
    assert lib.rc_session_info(ctypes.byref(n), ctypes.byref(d)) == OK and (n.value, d.value) == (R, -1)
    assert lib.rc_session_info(None, None) == OK


def test_struct_layouts_match_a_c_compiler(tmp_path):
    import subprocess
    from pathlib import Path
    root = Path(__file__).resolve().parent.parent
    structs = {"rc_route_desc": rows.RcRouteDesc, "rc_exchange_desc": rows.RcExchangeDesc,
               "rc_embedding_desc": rows.RcEmbeddingDesc}
    lines = [f'printf("%zu ", sizeof({n}));' for n in structs]
    for n, s in structs.items():
        lines += [f'printf("%zu ", offsetof({n}, {f[0]}));' for f in s._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "rc.h"\nint main(void){' + "".join(lines) +
                   "return 0;}\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", f"-I{root / 'include'}", str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = [ctypes.sizeof(s) for s in structs.values()]
    for s in structs.values():
        want += [getattr(s, f[0]).offset for f in s._fields_]
    assert got == want


# ---------------------------------------------------------------- the binding

@pytest.fixture
def two():
    rr.reset()
    rr.register(2, validate_only=True)
    yield
    rr.reset()


def code_of(fn):
    with pytest.raises(rr.CollectiveError) as e:
        fn()
    return e.value.code


def passes_checks(fn):
    with pytest.raises(ValueError, match="CUDA"):
        fn()


def f(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_route(two):
    l = [f(3, 8), f(0, 8)]
    passes_checks(lambda: rr.route(l, 2))
    assert code_of(lambda: rr.route(l[:1], 2)) == INVAL
    assert code_of(lambda: rr.route([f(3, 8), f(3, 7)], 2)) == SHAPE
    assert code_of(lambda: rr.route([f(3, 8), f(8)], 2)) == SHAPE
    assert code_of(lambda: rr.route([f(3, 8), f(3, 8, dtype=torch.bfloat16)], 2)) == DTYPE
    assert code_of(lambda: rr.route([f(8, 3).t(), f(3, 8)], 2)) == INVAL
    assert code_of(lambda: rr.route(l, 2, score="max")) == INVAL
    assert code_of(lambda: rr.route(l, 2, group_by="sum")) == INVAL
    assert code_of(lambda: rr.route(l, 2, bias=f(7))) == SHAPE
    assert code_of(lambda: rr.route(l, 2, bias=f(8, dtype=torch.float64))) == DTYPE
    assert code_of(lambda: rr.route(l, 2, out=([f(3, 2), f(1, 2)], [i(3, 2), i(0, 2)]))) == SHAPE
    assert code_of(lambda: rr.route(l, 2, out=([f(3, 2), f(0, 2)], [i(3, 2), f(0, 2)]))) == DTYPE
    with pytest.raises(TypeError):
        rr.route([f(3, 8, dtype=torch.float64)] * 2, 2)
    passes_checks(lambda: rr.route_grad(l, [i(3, 2), i(0, 2)], [f(3, 2), f(0, 2)]))
    assert code_of(lambda: rr.route_grad(l, [i(3, 2), i(0, 3)], [f(3, 2), f(0, 2)])) == SHAPE
    assert code_of(lambda: rr.route_grad(l, [i(3, 2)], [f(3, 2), f(0, 2)])) == INVAL
    assert code_of(lambda: rr.route_grad(l, [i(3, 2), i(0, 2)], [f(3, 2), f(0, 2)], out=[f(3, 8), f(1, 8)])) == SHAPE


def plan_of(capacity=(4, 5)):
    ex = [i(3, 2), i(1, 2)]
    return rows.DispatchPlan(ex, [i(3, 2), i(1, 2)], [i(3), i(3)], [i(2), i(2)], 4, list(capacity))


def test_binding_exchange(two):
    ex = [i(3, 2), i(1, 2)]
    passes_checks(lambda: rr.dispatch_plan(ex, 4))
    assert code_of(lambda: rr.dispatch_plan(ex, 3)) == INVAL
    assert code_of(lambda: rr.dispatch_plan(ex, 0)) == INVAL
    assert code_of(lambda: rr.dispatch_plan(ex, 4, capacity=[1])) == INVAL
    assert code_of(lambda: rr.dispatch_plan([i(3, 2), i(1, 3)], 4)) == SHAPE
    assert code_of(lambda: rr.dispatch_plan([i(3, 2), f(1, 2)], 4)) == DTYPE
    p = plan_of()
    x, y = [f(3, 8), f(1, 8)], [f(4, 8), f(5, 8)]
    w = [f(3, 2), f(1, 2)]
    passes_checks(lambda: rr.dispatch(x, p))
    passes_checks(lambda: rr.combine(y, p))
    passes_checks(lambda: rr.combine(y, p, w))
    passes_checks(lambda: rr.combine_grad(x, y, p, w))
    assert code_of(lambda: rr.dispatch([f(3, 8), f(2, 8)], p)) == SHAPE
    assert code_of(lambda: rr.dispatch(x, p, out=[f(4, 8), f(4, 8)])) == SHAPE
    assert code_of(lambda: rr.dispatch(x, p, out=[f(4, 8), f(5, 8, dtype=torch.float16)])) == DTYPE
    assert code_of(lambda: rr.combine([f(4, 8), f(4, 8)], p)) == SHAPE
    assert code_of(lambda: rr.combine(y, p, [f(3, 2), f(1, 1)])) == SHAPE
    assert code_of(lambda: rr.combine(y, p, out=x[:1])) == INVAL
    assert code_of(lambda: rr.combine_grad(x, [f(4, 8), f(5, 7)], p, w)) == SHAPE
    p.slots[1] = i(1, 3)
    assert code_of(lambda: rr.dispatch(x, p)) == SHAPE


def test_binding_embedding(two):
    ids = [i(3), i(0)]
    passes_checks(lambda: rr.embedding(ids, [f(3, 8), f(2, 8)]))
    assert code_of(lambda: rr.embedding(ids, [f(2, 8), f(3, 8)])) == SHAPE  # not the segments of 5
    assert code_of(lambda: rr.embedding(ids, [f(3, 8)])) == INVAL
    assert code_of(lambda: rr.embedding([i(3), f(0)], [f(3, 8), f(2, 8)])) == DTYPE
    assert code_of(lambda: rr.embedding([i(3, 1), i(0)], [f(3, 8), f(2, 8)])) == SHAPE
    with pytest.raises(TypeError):
        rr.embedding([f(3), f(0)], [f(3, 8), f(2, 8)])
    d = [f(3, 8), f(0, 8)]
    passes_checks(lambda: rr.embedding_grad(ids, d, 5))
    assert code_of(lambda: rr.embedding_grad(ids, d, 5, accumulate=True)) == INVAL
    assert code_of(lambda: rr.embedding_grad(ids, d, 5, out=[f(3, 8), f(3, 8)])) == SHAPE
    assert code_of(lambda: rr.embedding_grad(ids, [f(2, 8), f(0, 8)], 5)) == SHAPE
    assert code_of(lambda: rr.embedding_grad(ids, d, 5, dtype=torch.float16, out=[f(3, 8), f(2, 8)])) == DTYPE
    assert rows.shard_rows(5, 4) == [2, 2, 1, 0]


def test_binding_sizes(two):
    """Outputs too large for any buffer are refused before they are allocated."""
    x = [f(3, 8), f(1, 8)]
    for capacity in ((2**31, 5), (2**62, 2**62), (2**63 - 1, 0)):
        assert code_of(lambda: rr.dispatch(x, plan_of(capacity))) == INVAL
    assert code_of(lambda: rr.combine([f(0, 2**40)] * 2, plan_of((0, 0)))) == INVAL
    for vocab in (0, -1, 2**31, 2**62, 2**63 - 1):
        assert code_of(lambda: rr.embedding_grad([i(3), i(0)], [f(3, 8), f(0, 8)], vocab)) == INVAL
