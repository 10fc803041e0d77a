"""Block operators on the CPU: the oracle against differences, and every refusal
of the C ABI (validate_only sessions, fake addresses) and of the binding (host
tensors)."""

import ctypes

import numpy as np
import pytest
import torch

import rank_reductions_amd as rr
from oracle import blocks as orc
from rank_reductions_amd import blocks
from test_rows_cpu import INVAL, NR, OK, R, Space, lib, ptrs  # noqa: F401

F32, F16, BF16, E4M3 = 0, 2, 3, 5
DTYPE, SHAPE = rr.RC_ERR_DTYPE_MISMATCH, rr.RC_ERR_SHAPE_MISMATCH


# ---------------------------------------------------------------- the oracle

def test_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    s, w, dy, ds = rng.normal(size=(3, 7)), rng.normal(size=7), rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    dx, dw = orc.rms_norm_grad(dy, s, w, 0.1, ds)

    def loss(s, w):
        return (orc.rms_norm(s, w, 0.1)[0] * dy).sum() + (s * ds).sum()

    h = 1e-6
    for t in range(3):
        for i in range(7):
            e = np.zeros_like(s)
            e[t, i] = h
            assert abs((loss(s + e, w) - loss(s - e, w)) / (2 * h) - dx[t, i]) < 1e-8
    for i in range(7):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((loss(s, w + e) - loss(s, w - e)) / (2 * h) - dw[i]) < 1e-8


def test_adamw_by_hand():
    p, m, v = orc.adamw([1.0], [2.0], [0.0], [0.0], 1, lr=0.1, betas=(0.9, 0.99), eps=0.0, weight_decay=0.5)
    assert abs(m[0] - 0.2) < 1e-15 and abs(v[0] - 0.04) < 1e-15
    assert abs(p[0] - (1 - 0.05 - 0.1)) < 1e-12  # the first step's update is the gradient's sign


def test_8bit_codes_of_means():
    """Codes to nearest against torch's own, and those by chance: no more than a step away, right on the average."""
    rng = np.random.default_rng(2)
    x = np.concatenate([rng.normal(size=4000) * 10.0 ** rng.integers(-4, 3, size=4000), [0, 448, 460, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]])
    near = torch.tensor(np.clip(x, -448, 448), dtype=torch.float64).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(orc.e4m3(x), near)
    c, held = orc.mean_codes(x, np.ones_like(x), 1.0, 0.9, 0.5)
    assert np.array_equal(c, near) and not held.any()
    # 0.9 k rounds to k for one to four of the smallest codes; 0.95 k up to ten, and for nine and ten eighths of the 14
    # octaves above; 0.99 k for all
    k = np.unique(orc.e4m3(2.0 ** np.linspace(-9, 8.8, 2000)))
    for beta, kept in ((0.9, 4), (0.95, 10 + 2 * 14), (0.99, k.size)):
        stays = orc.e4m3(beta * k) == k
        assert stays.sum() == kept and not (stays & ~orc.mean_codes(beta * k, 0 * k, 1.0, beta, 0.5)[1]).any()
    y = np.full(1 << 16, -3.6 * 2.0 ** -9)
    c, held = orc.mean_codes(y, np.zeros_like(y), 1.0, 0.9, np.arange(1 << 16) / 65536)
    assert held.all() and set(c * 512) == {-4.0, -3.0} and abs(c.mean() / y[0] - 1) < 1e-4


@pytest.mark.parametrize("beta1", [0.9, 0.95, 0.99])
@pytest.mark.parametrize("steady", [True, False])
@pytest.mark.parametrize("tiny", [0.0, 1e-9])
def test_8bit_means_without_a_gradient_go(beta1, steady, tiny):
    """Half a block loses its gradient after 20 steps (or keeps next to none of it); the rest go on, one of them with a
    steady gradient that holds the scale.  To nearest the idle means would stay, and their parameters drift by up to
    the rate and far more in every step.  By chance a mean of up to 2^18 of the smallest codes decays on the average as
    it should, and is gone when that falls to 2^-18 codes: ln(2^36) / (1 - beta1) < 25 / (1 - beta1) steps on (a
    chance of 256 * 2^-18 that one is left).  Its parameter stays from then on.  With 1e-9 of a gradient a mean may
    now and then be one smallest code: 8 / 448 * 2^-9 at most, over a root whose square is 0.02 of the mean of twenty
    squares, 0.3 or more, and decays by 0.999 a step; twice that for the root's own rounding."""
    rng = np.random.default_rng(5)
    idle = np.arange(256) % 2 == 1
    state = np.zeros(256), np.zeros(256), 0.0, np.zeros(256), 0.0
    gone = 20 + int(25 / (1 - beta1))
    for t in range(1, gone + 2001):
        g = rng.normal(size=256)
        if t > 20:
            g[idle] *= tiny
        if steady:
            g[0] = 8.0
        state = orc.adamw8(state[0], g, *state[1:], t, weight_decay=0.0, betas=(beta1, 0.999))
        if t == gone:
            rest = state[0][idle]
    assert (np.abs(state[1][idle]) <= (2.0 ** -9 if tiny else 0)).all() and state[1][~idle].any()
    moved = np.abs(state[0][idle] - rest).max()
    assert moved <= (2 * 2000 * 1e-3 * 8 / 448 * 2.0 ** -9 / (0.02 * 0.3 * 0.999 ** t) ** 0.5 if tiny else 0)


def test_adamw_follows_torch():
    rng = np.random.default_rng(1)
    x = torch.tensor(rng.normal(size=40), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([x], lr=0.01, betas=(0.8, 0.9), eps=1e-3, weight_decay=0.1)
    p, m, v = x.detach().numpy().copy(), np.zeros(40), np.zeros(40)
    for t in range(1, 5):
        g = rng.normal(size=40)
        x.grad = torch.tensor(g)
        opt.step()
        p, m, v = orc.adamw(p, g, m, v, t, 0.01, (0.8, 0.9), 1e-3, 0.1)
        assert np.allclose(p, x.detach().numpy(), rtol=1e-12, atol=0)


def test_largest_of_groups():
    y = np.array([[1.0, -3.0, 2.0, 0.5, -0.25]])
    assert orc.largest(y).tolist() == [[3.0]] and orc.largest(y, 2).tolist() == [[3.0, 2.0, 0.25]]


# ---------------------------------------------------------------- the C ABI: norm

def norm_args(grad=False, **kw):
    o = dict(dtype=F32, weight_dtype=F32, quantize=0, group=0, eps=1e-6, width=64, size=None, tokens=[3] * R, residual=True,
             drop=None, shift=None, same=None, ws=None)
    o.update(kw)
    tokens = (ctypes.c_int64 * R)(*o["tokens"])
    d = blocks.RcNormDesc()
    d.struct_size = ctypes.sizeof(d) if o["size"] is None else o["size"]
    for k in ("dtype", "weight_dtype", "quantize", "group", "eps", "width"):
        setattr(d, k, o[k])
    d.tokens = ctypes.addressof(tokens)
    sp = Space()
    n = 1 << 22
    names = ["d_ys", "sums", "weights", "d_sums", "d_xs", "d_weights"] if grad else ["xs", "residuals", "weights", "ys", "scales", "sums"]
    bufs = {k: [sp.take(n) for _ in range(R)] for k in names}
    if o["drop"]:
        bufs[o["drop"][0]][o["drop"][1]] = None
    if o["shift"]:
        bufs[o["shift"][0]][1] += o["shift"][1]
    if o["same"]:
        bufs[o["same"][0]][2] = bufs[o["same"][1]][2] + (o["same"][2] if len(o["same"]) > 2 else 0)
    arrays = {k: ptrs(v) for k, v in bufs.items()}
    if not o["residual"]:
        for k in ("residuals", "sums") if not grad else ("d_sums",):
            arrays[k] = None
    for k in o.get("null", ()):
        arrays[k] = None
    args = [ctypes.byref(d)] + [arrays[k] for k in names]
    if grad:
        ws = 1 << 24 if o["ws"] is None else o["ws"]
        args += [ctypes.c_void_p(sp.take(1 << 24)), ws]
    return args + [None], (d, tokens, arrays)


NORM_OK = [dict(), dict(residual=False), dict(dtype=BF16), dict(dtype=F16, weight_dtype=F16), dict(width=1), dict(width=32768),
           dict(tokens=[0] * R), dict(tokens=[0, 5, 0, 1], drop=("xs", 0)), dict(quantize=1, dtype=BF16), dict(quantize=1, group=128),
           dict(eps=0.0), dict(same=("sums", "residuals")), dict(same=("ys", "xs"))]
NORM_BAD = [dict(size=8), dict(dtype=1), dict(dtype=E4M3), dict(weight_dtype=BF16), dict(width=0), dict(width=32769), dict(eps=-1.0),
            dict(eps=float("nan")), dict(eps=float("inf")), dict(quantize=2), dict(group=16), dict(group=512), dict(group=-1),
            dict(tokens=[-1, 0, 0, 0]), dict(tokens=[2**31 - 1, 1, 0, 0]), dict(drop=("xs", 1)), dict(drop=("weights", 0)),
            dict(drop=("sums", 3)), dict(shift=("xs", 2)), dict(shift=("sums", 1)), dict(same=("ys", "weights")),
            dict(same=("sums", "xs", 4)), dict(same=("sums", "residuals", 4)), dict(same=("ys", "sums")), dict(null=("weights",)),
            dict(null=("sums",)), dict(null=("residuals",)), dict(quantize=1, null=("scales",)), dict(quantize=1, same=("ys", "xs"))]


@pytest.mark.parametrize("kw", NORM_OK, ids=str)
def test_norm_accepts(lib, kw):  # noqa: F811
    args, keep = norm_args(**kw)
    assert lib.rc_rms_norm(*args) == OK, lib.rc_last_error()


@pytest.mark.parametrize("kw", NORM_BAD, ids=str)
def test_norm_refuses(lib, kw):  # noqa: F811
    args, keep = norm_args(**kw)
    assert lib.rc_rms_norm(*args) == INVAL
    assert b"rms_norm" in lib.rc_last_error()


@pytest.mark.parametrize("kw", [dict(), dict(residual=False), dict(dtype=BF16), dict(tokens=[0] * R), dict(same=("d_xs", "d_ys")),
                                dict(same=("d_xs", "d_sums"))], ids=str)
def test_norm_grad_accepts(lib, kw):  # noqa: F811
    args, keep = norm_args(grad=True, **kw)
    assert lib.rc_rms_norm_grad(*args) == OK, lib.rc_last_error()


@pytest.mark.parametrize("kw", [dict(width=0), dict(ws=0), dict(ws=R * 3 * 64 * 4 - 1), dict(drop=("d_weights", 0)), dict(drop=("d_sums", 0)),
                                dict(same=("d_xs", "sums")), dict(same=("d_weights", "weights")), dict(same=("d_xs", "d_ys", 4)),
                                dict(null=("d_ys",)), dict(shift=("d_weights", 2))], ids=str)
def test_norm_grad_refuses(lib, kw):  # noqa: F811
    args, keep = norm_args(grad=True, **kw)
    assert lib.rc_rms_norm_grad(*args) == INVAL
    assert b"rms_norm_grad" in lib.rc_last_error()


def test_norm_grad_workspace(lib):  # noqa: F811
    args, (d, *keep) = norm_args(grad=True)
    size = ctypes.c_int64()
    assert lib.rc_rms_norm_grad_workspace(args[0], ctypes.byref(size)) == OK
    assert size.value == R * 3 * 64 * 4  # a workgroup for each of a few tokens
    assert lib.rc_rms_norm_grad_workspace(args[0], None) == INVAL


# ---------------------------------------------------------------- experts

def moe_args(**kw):
    o = dict(dtype=BF16, weight_dtype=BF16, out_dtype=BF16, num_experts=8, top_k=2, width=64, inner=32, size=None, tokens=[3] * R, drop=None,
             shift=None, same=None, ws=1 << 24, scales=None, weight_scales=None, null=())
    o.update(kw)
    tokens = (ctypes.c_int64 * R)(*o["tokens"])
    d = blocks.RcMoeDesc()
    d.struct_size = ctypes.sizeof(d) if o["size"] is None else o["size"]
    for k in ("dtype", "weight_dtype", "out_dtype", "num_experts", "top_k", "width", "inner"):
        setattr(d, k, o[k])
    d.tokens = ctypes.addressof(tokens)
    sp = Space()
    names = ["xs", "scales", "experts", "weights", "gate_up", "gate_up_scales", "down", "down_scales", "ys"]
    bufs = {k: [sp.take(1 << 24) for _ in range(R)] for k in names}
    if o["drop"]:
        bufs[o["drop"][0]][o["drop"][1]] = None
    if o["shift"]:
        bufs[o["shift"][0]][1] += o["shift"][1]
    if o["same"]:
        bufs[o["same"][0]][2] = bufs[o["same"][1]][2]
    arrays = {k: ptrs(v) for k, v in bufs.items()}
    eight = o["dtype"] == E4M3 if o["scales"] is None else o["scales"]
    weights8 = o["weight_dtype"] == E4M3 if o["weight_scales"] is None else o["weight_scales"]
    if not eight:
        arrays["scales"] = None
    if not weights8:
        arrays["gate_up_scales"] = arrays["down_scales"] = None
    for k in o["null"]:
        arrays[k] = None
    return [ctypes.byref(d)] + [arrays[k] for k in names] + [ctypes.c_void_p(sp.take(1 << 25)), o["ws"], None], (d, tokens, arrays)


MOE_OK = [dict(), dict(dtype=F32, weight_dtype=F32, out_dtype=F32), dict(weight_dtype=E4M3), dict(dtype=E4M3, weight_dtype=E4M3),
          dict(dtype=E4M3, weight_dtype=E4M3, out_dtype=F32), dict(tokens=[0] * R, ws=0), dict(tokens=[256] * R, width=1, inner=1),
          dict(num_experts=1024), dict(width=1, inner=1, top_k=1), dict(top_k=16, tokens=[32] * R)]
MOE_BAD = [dict(size=8), dict(dtype=1), dict(weight_dtype=F16), dict(dtype=F32, weight_dtype=E4M3, out_dtype=F32), dict(out_dtype=F32),
           dict(dtype=E4M3), dict(dtype=E4M3, weight_dtype=E4M3, out_dtype=E4M3), dict(num_experts=0), dict(num_experts=6),
           dict(num_experts=1028), dict(top_k=0), dict(top_k=17), dict(width=0), dict(width=65537), dict(inner=0), dict(inner=65537),
           dict(tokens=[257, 256, 256, 256]), dict(tokens=[-1, 0, 0, 0]), dict(ws=100), dict(drop=("xs", 0)), dict(drop=("gate_up", 3)),
           dict(drop=("down", 0)), dict(drop=("weights", 1)), dict(shift=("xs", 1)), dict(shift=("experts", 2)), dict(same=("ys", "xs")),
           dict(same=("ys", "down")), dict(null=("xs",)), dict(null=("experts",)), dict(null=("gate_up",)), dict(null=("ys",)),
           dict(scales=True), dict(weight_scales=True), dict(weight_dtype=E4M3, weight_scales=False),
           dict(weight_dtype=E4M3, null=("down_scales",)), dict(dtype=E4M3, weight_dtype=E4M3, scales=False)]


@pytest.mark.parametrize("kw", MOE_OK, ids=str)
def test_moe_accepts(lib, kw):  # noqa: F811
    args, keep = moe_args(**kw)
    assert lib.rc_moe_layer(*args) == OK, lib.rc_last_error()


@pytest.mark.parametrize("kw", MOE_BAD, ids=str)
def test_moe_refuses(lib, kw):  # noqa: F811
    args, keep = moe_args(**kw)
    assert lib.rc_moe_layer(*args) == INVAL
    assert b"moe_layer" in lib.rc_last_error()


def test_moe_workspace(lib):  # noqa: F811
    args, (d, *keep) = moe_args(width=100, inner=65)
    size = ctypes.c_int64()
    assert lib.rc_moe_layer_workspace(args[0], ctypes.byref(size)) == OK
    assert size.value == 24 * (128 + 112) * 4 + 8 * 16 + 48


@pytest.mark.parametrize("out,each", [(F32, 6), (BF16, 4), (F16, 4)])
def test_moe_workspace_of_8bit_rows(lib, out, each):  # noqa: F811
    """Float32 outputs need a third number for each hidden value; one byte less is refused."""
    args, (d, *keep) = moe_args(width=100, inner=65, dtype=E4M3, weight_dtype=E4M3, out_dtype=out)
    size = ctypes.c_int64()
    assert lib.rc_moe_layer_workspace(args[0], ctypes.byref(size)) == OK
    assert size.value == 24 * (128 * each + 112 * 4) + 8 * 16 + 48
    for less, code in ((0, OK), (1, INVAL)):
        args[-2] = size.value - less
        assert lib.rc_moe_layer(*args) == code, lib.rc_last_error()


# ---------------------------------------------------------------- gradients and steps

def grads_of(sp, counts, dtype=F32):
    arr = (blocks.RcGrad * max(1, len(counts)))()
    for g, n in zip(arr, counts):
        g.grad, g.count, g.dtype = (sp.take(n * 4 + 64) if n else None), n, dtype
    return arr


def lists_of(arrays):
    return ptrs([ctypes.addressof(a) for a in arrays])


def grad_norm(lib, edit=None, ws=None, size=None, norms=True):  # noqa: F811
    sp = Space()
    arrays = [grads_of(sp, [10, 0, 70000], dt) for dt in (F32, BF16, F16, F32)]
    if edit:
        edit(arrays)
    d = blocks.RcGradNormDesc()
    d.struct_size = ctypes.sizeof(d) if size is None else size
    counts = (ctypes.c_int * R)(3, 3, 3, 3)
    need = ctypes.c_int64()
    status = lib.rc_grad_norm_workspace(ctypes.byref(d), counts, lists_of(arrays), ctypes.byref(need))
    if status != OK:
        return status
    return lib.rc_grad_norm(ctypes.byref(d), counts, lists_of(arrays), ctypes.c_void_p(sp.take(64) if norms else None),
                            ctypes.c_void_p(sp.take(1 << 20)), need.value if ws is None else ws, None)


def test_grad_norm_accepts_and_refuses(lib):  # noqa: F811
    assert grad_norm(lib) == OK, lib.rc_last_error()

    def change(field, value, at=0):
        def edit(arrays):
            setattr(arrays[1][at], field, value)
        return edit

    assert grad_norm(lib, change("grad", None, 1)) == OK
    for edit in (change("dtype", 1), change("dtype", E4M3), change("count", -1), change("count", 1 << 39), change("grad", None),
                 change("grad", (1 << 33) + 1), change("grad", 1 << 60)):
        assert grad_norm(lib, edit) == INVAL, "accepted"
        assert b"grad_norm" in lib.rc_last_error()
    assert grad_norm(lib, ws=8) == INVAL and grad_norm(lib, size=4) == INVAL and grad_norm(lib, norms=False) == INVAL


class Steps:
    """Tables of two states, and a step by them."""

    def __init__(self, lib, bits=32, dtype=BF16, counts=(300, 0, 9000)):  # noqa: F811
        self.lib, self.bits, self.sp = lib, bits, Space()
        self.counts = counts
        self.n = (ctypes.c_int * R)(*[len(counts)] * R)
        self.params = [self.make(dtype) for _ in range(2)]
        self.grads = [grads_of(self.sp, counts, F32) for _ in range(R)]
        self.steps, self.out_steps, self.norms, self.lr = (self.sp.take(64) for _ in range(4))
        self.gpu = [self.sp.take(1 << 20) for _ in range(2)]
        self.tables = [None, None]

    def make(self, dtype):
        out = []
        for _ in range(R):
            arr = (blocks.RcAdamwParam * len(self.counts))()
            for p, n in zip(arr, self.counts):
                p.count, p.dtype = n, dtype
                for k in ("param", "master", "m", "v", "m_scale", "v_scale"):
                    setattr(p, k, self.sp.take(n * 4 + 64))
            out.append(arr)
        return out

    def table(self, which=0, size=None, bits=None, session=0, room=None):
        d = blocks.RcAdamwTableDesc()
        d.struct_size = ctypes.sizeof(d) if size is None else size
        d.state_bits = self.bits if bits is None else bits
        d.session = session
        n = ctypes.c_int64()
        args = [ctypes.byref(d), self.n, lists_of(self.params[which])]
        status = self.lib.rc_adamw_table(*args, None, ctypes.byref(n))
        if status != OK:
            return status
        self.tables[which] = (ctypes.c_uint64 * (n.value // 8 + 1))()
        if room is not None:
            n.value = room
        return self.lib.rc_adamw_table(*args, self.tables[which], ctypes.byref(n))

    def step(self, out=0, gpu=None, size=None, table=None, **kw):
        d = blocks.RcAdamwDesc()
        d.struct_size = ctypes.sizeof(d) if size is None else size
        d.lr, d.beta1, d.beta2, d.eps, d.weight_decay, d.grad_scale = 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0
        d.steps = d.steps_out = self.steps
        for k, v in kw.items():
            setattr(d, k, v)
        t = self.tables[0] if table is None else table
        return self.lib.rc_adamw_step(ctypes.byref(d), t, ctypes.c_void_p(self.gpu[0]), self.tables[out],
                                      ctypes.c_void_p(self.gpu[out] if gpu is None else gpu), lists_of(self.grads), None)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_step_accepts(lib, bits, dtype):  # noqa: F811
    s = Steps(lib, bits, dtype)
    assert s.table(0) == OK and s.table(1) == OK, lib.rc_last_error()
    assert s.step() == OK, lib.rc_last_error()
    assert s.step(out=1, steps_out=s.out_steps) == OK, lib.rc_last_error()
    assert s.step(norms=s.norms, max_norm=1.0, lr_on_gpu=s.lr) == OK
    for g in s.grads[2]:
        g.grad, g.count = None, 0
    assert s.step() == OK
    if dtype != F32:
        s.grads[0][0].dtype = dtype
        assert s.step() == OK


def test_table_refuses(lib):  # noqa: F811
    def fresh(**kw):
        return Steps(lib, **kw)

    assert fresh().table(bits=16) == INVAL and fresh().table(size=4) == INVAL and fresh().table(room=64) == INVAL
    assert fresh().table(session=12345) == INVAL
    for k, v in (("count", -1), ("count", 1 << 39), ("dtype", 1), ("param", None), ("master", None), ("m", None), ("v", None)):
        s = fresh()
        setattr(s.params[0][1][0], k, v)
        assert s.table() == INVAL, k
        assert b"adamw_table" in lib.rc_last_error()
    for k in ("m_scale", "v_scale"):
        s = fresh(bits=8)
        setattr(s.params[0][0][2], k, None)
        assert s.table() == INVAL
    s = fresh()
    s.params[0][1][0].m = s.params[0][3][2].v + 4
    assert s.table() == INVAL and b"overlap" in lib.rc_last_error()
    s = fresh()
    s.n[2] = -1
    assert s.table() == INVAL
    # float32 parameters have no copies, states of 32 bits no scales
    s = fresh(dtype=F32)
    for a in s.params[0]:
        for p in a:
            p.master = p.m_scale = p.v_scale = None
    assert s.table() == OK


@pytest.mark.parametrize("out", [0, 1])
def test_step_refuses_tables_among_its_buffers(lib, out):  # noqa: F811
    """A table on the GPU that lies in a parameter's buffer would be stepped over while kernels go by it; gradients that
    the step writes before it reads them."""
    for which in range(out + 1):
        for k in ("param", "master", "m", "v"):
            s = Steps(lib)
            assert s.table(0) == OK and s.table(1) == OK
            s.gpu[which] = getattr(s.params[which][1][2], k) + 64 & ~15
            assert s.step(out=out, steps_out=s.out_steps) == INVAL, (which, k)
            assert b"overlap" in lib.rc_last_error()
        s = Steps(lib)
        s.gpu[0] = s.params[which][0][0].v & ~15
        assert s.table(0) == OK and s.table(1) == OK
        assert s.step(out=out, steps_out=s.out_steps) == INVAL
    for at in ("gpu", "out_steps"):
        s = Steps(lib)
        assert s.table(0) == OK and s.table(1) == OK
        s.grads[1][2].grad = s.gpu[0] + 512 if at == "gpu" else s.out_steps + 4
        assert s.step(out=out, steps_out=s.out_steps) == INVAL, at
        assert b"gradient 2: overlaps" in lib.rc_last_error()


def test_step_refuses(lib):  # noqa: F811
    s = Steps(lib)
    assert s.table(0) == OK and s.table(1) == OK
    nan, inf = float("nan"), float("inf")
    for kw in (dict(size=4), dict(lr=-1.0), dict(lr=nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan), dict(beta2=1.0), dict(eps=-1e-9),
               dict(eps=inf), dict(weight_decay=nan), dict(max_norm=1.0), dict(norms=s.norms, max_norm=-1.0), dict(grad_scale=inf),
               dict(steps=None), dict(steps_out=None), dict(norms=s.norms + 2), dict(lr_on_gpu=s.lr + 1), dict(steps_out=s.steps + 4),
               dict(norms=s.steps), dict(gpu=s.gpu[1]), dict(gpu=s.gpu[0] + 8), dict(out=1, gpu=s.gpu[0]),
               dict(steps_out=s.params[0][0][0].m, steps=s.params[0][0][0].m), dict(norms=s.params[0][1][0].param),
               dict(session=999)):
        assert s.step(**kw) == INVAL, kw
        assert b"adamw_step" in lib.rc_last_error()
    # max_norm may be infinite: no bound
    assert s.step(norms=s.norms, max_norm=inf) == OK
    for k, v in (("count", 299), ("dtype", F16), ("grad", None), ("grad", s.params[0][2][2].v + 8)):
        t = Steps(lib)
        assert t.table(0) == OK and t.table(1) == OK
        setattr(t.grads[1][0], k, v)
        if k == "grad" and v is not None:
            t.grads[1][0].grad = t.params[0][2][2].v + 8
        assert t.step() == INVAL, (k, v)
    # another state's buffers
    t = Steps(lib)
    t.params[1][3][0].m = t.params[0][0][2].v
    assert t.table(0) == OK and t.table(1) == OK and t.step(out=1, steps_out=t.out_steps) == INVAL and b"share" in lib.rc_last_error()
    t = Steps(lib)
    t.params[1] = t.make(F32)
    assert t.table(0) == OK and t.table(1) == OK and t.step(out=1) == INVAL and b"differ" in lib.rc_last_error()
    junk = (ctypes.c_uint64 * 4096)()
    assert s.step(table=junk) == INVAL


def test_without_a_session_and_after_it(lib):  # noqa: F811
    s = Steps(lib)
    assert s.table(0) == OK
    args, keep = norm_args()
    moe, keep2 = moe_args()
    lib.rc_reset()
    assert lib.rc_rms_norm(*args) == NR and lib.rc_moe_layer(*moe) == NR and s.step() == NR and grad_norm(lib) == NR
    cfg = rr.make_config(validate_only=True)
    assert lib.rc_register(R // 2, ctypes.byref(cfg)) == OK
    assert s.step() == INVAL and b"ranks" in lib.rc_last_error()
    for d in (keep[0], keep2[0]):
        d.session = 1
    assert lib.rc_rms_norm(*args) == INVAL and b"closed" in lib.rc_last_error()
    assert lib.rc_moe_layer(*moe) == INVAL and b"closed" in lib.rc_last_error()


# ---------------------------------------------------------------- the binding

@pytest.fixture
def two():
    rr.library().rc_reset()
    cfg = rr.make_config(validate_only=True)
    assert rr.library().rc_register(2, ctypes.byref(cfg)) == OK
    yield
    rr.library().rc_reset()


def code(fn, *args, **kw):
    with pytest.raises((rr.CollectiveError, TypeError, ValueError)) as e:
        fn(*args, **kw)
    return getattr(e.value, "status", None) or getattr(e.value, "code", None) or type(e.value)


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_norms(two):
    x, w = [z(2, 8), z(1, 8)], [z(8), z(8)]
    for args, kw in (((x[:1], w), {}), ((x, w[:1]), {}), (([z(2, 8), z(1, 9)], w), {}), (([z(2), z(1)], w), {}), ((x, [z(9), z(9)]), {}),
                     ((x, [z(8, dtype=torch.float16)] * 2), {}), ((x, w), dict(residuals=x[:1])), ((x, w), dict(quantize="int8")),
                     ((x, w), dict(residuals=x, out=x)), ((x, w), dict(quantize="e4m3", out=(x, x))), (("xy", w), {}),
                     (([z(8, 2).t(), z(1, 8)], w), {}), (([None, None], w), {}), ((x, w), {})):
        code(rr.rms_norm, *args, **kw)  # the last for tensors that are not on a GPU
    code(rr.rms_norm, [z(2, 8, dtype=torch.int32)] * 2, w)
    for args, kw in (((x, x, w), {}), ((x[:1], x, w), {}), ((x, x, w), dict(d_sums=[z(2, 8), z(2, 8)])), ((x, x, w), dict(out=x[0]))):
        code(rr.rms_norm_grad, *args, **kw)


def test_binding_refuses_layers(two):
    x, w, e = [z(2, 8), z(1, 8)], [z(2, 2), z(1, 2)], [z(2, 2, dtype=torch.int32), z(1, 2, dtype=torch.int32)]
    gu, dn = [z(2, 6, 8)] * 2, [z(2, 8, 3)] * 2
    for args, kw in (((x, w, e, gu, dn), {}), ((x, w, w, gu, dn), {}), ((x, e, e, gu, dn), {}), ((x, w, e, [z(2, 5, 8)] * 2, dn), {}),
                     ((x, w, e, gu, [z(2, 8, 4)] * 2), {}), ((x, w, e, [z(6, 8)] * 2, dn), {}), ((x, w, e, gu, dn[:1]), {}),
                     ((x, w, e, gu, dn), dict(dtype="f32")), ((x, w, e, gu, dn), dict(scales=[z(2, 2), z(1, 2)])),
                     ((x, w, e, gu, dn), dict(gate_up_scales=[z(2, 5)] * 2)), ((x, w, e, gu, dn), dict(out=x[:1])),
                     ((x, w, e, [g.half() for g in gu], dn), {})):
        code(rr.moe_layer, *args, **kw)


def test_binding_refuses_steps(two):
    p = [{0: z(5)}, {0: z(5)}]
    code(rr.adamw_state, p)  # not on a GPU
    code(rr.adamw_state, [{}, {}])
    code(rr.adamw_state, p[:1])
    code(rr.adamw_state, p, bits=16)
    code(rr.AdamWState, p, 32, [{}, {}], p, z(2, dtype=torch.int32))
    code(rr.AdamWState, [{0: z(5).half()}] * 2, 32, p, p, z(2, dtype=torch.int32))
    code(rr.grad_norm, p)
    code(rr.grad_norm, p, over="some")
    code(rr.grad_norm, [{}, {}])
    code(rr.grad_norm, [{0: 1.0}, {}])
    code(rr.grad_norm, [[z(3)], {}])


def test_struct_layouts_match_a_c_compiler(tmp_path):
    import subprocess
    from pathlib import Path

    structs = {"rc_norm_desc": blocks.RcNormDesc, "rc_moe_desc": blocks.RcMoeDesc, "rc_grad": blocks.RcGrad,
               "rc_grad_norm_desc": blocks.RcGradNormDesc, "rc_adamw_table_desc": blocks.RcAdamwTableDesc,
               "rc_adamw_param": blocks.RcAdamwParam, "rc_adamw_desc": blocks.RcAdamwDesc}
    lines, want = [], []
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {field}));')
            want.append(getattr(cls, field).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "rc.h"\nint main(void){' + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "layout"
    include = Path(__file__).resolve().parent.parent / "include"
    subprocess.run(["gcc", f"-I{include}", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in out.split()] == want
