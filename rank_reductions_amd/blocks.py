"""Block operators: what stands around a mixture-of-experts block and behind a
gradient sync (whole-call form; include/rc.h, "Block operators").

    ys, sums = rr.rms_norm(xs, weights, residuals=hs)      # R tensors each
    codes, scales, sums = rr.rms_norm(xs, weights, residuals=hs, quantize="e4m3")
    d_xs, d_weights = rr.rms_norm_grad(d_ys, sums, weights, d_sums=d_hs)

    weights, experts = rr.route(logits, top_k=8)
    ys = rr.moe_layer(xs, weights, experts, gate_up, down) # a few tokens, no dispatch

    state = rr.adamw_state(params, bits=8)                 # params[r]: {id: tensor}
    rr.all_reduce_params(grads, "mean", out=grads)
    norms = rr.grad_norm(grads)
    rr.adamw_step(state, grads, lr=1e-3, norms=norms, max_norm=1.0)

Argument marshalling only, as of the row exchanges (rows.py): tensors are given
as one per rank, on the session's GPU; new ones are allocated, and kernels
enqueued, on `stream` (the current one if None), and the parts of one call may
share an allocation.
"""

import ctypes

import rank_reductions_amd as _rr
from rank_reductions_amd.rows import _call, _choice

__all__ = ["rms_norm", "rms_norm_grad", "moe_layer", "grad_norm", "AdamWState", "adamw_state", "adamw_step"]


RC_E4M3 = 5
QUANTIZE = {None: 0, "e4m3": 1}


class RcNormDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("quantize", ctypes.c_int32),
        ("group", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("width", ctypes.c_int64),
        ("tokens", ctypes.c_void_p),
        ("session", ctypes.c_int64),
    ]


class RcMoeDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("width", ctypes.c_int64),
        ("inner", ctypes.c_int64),
        ("tokens", ctypes.c_void_p),
        ("session", ctypes.c_int64),
    ]


class RcGrad(ctypes.Structure):
    _fields_ = [
        ("grad", ctypes.c_void_p),
        ("count", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class RcGradNormDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("over_all", ctypes.c_int32),
        ("session", ctypes.c_int64),
    ]


class RcAdamwTableDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("state_bits", ctypes.c_int32),
        ("session", ctypes.c_int64),
    ]


class RcAdamwParam(ctypes.Structure):
    _fields_ = [
        ("count", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("param", ctypes.c_void_p),
        ("master", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
    ]


class RcAdamwDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("seed", ctypes.c_uint32),
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
        ("max_norm", ctypes.c_double),
        ("grad_scale", ctypes.c_double),
        ("lr_on_gpu", ctypes.c_void_p),
        ("norms", ctypes.c_void_p),
        ("steps", ctypes.c_void_p),
        ("steps_out", ctypes.c_void_p),
        ("session", ctypes.c_int64),
    ]


def declare(lib):
    """Argument types of the library's block operators."""
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name, args in {
        "rc_rms_norm": [p, p, p, p, p, p, p, p],
        "rc_rms_norm_grad_workspace": [p, p],
        "rc_rms_norm_grad": [p, p, p, p, p, p, p, p, i64, p],
        "rc_moe_layer_workspace": [p, p],
        "rc_moe_layer": [p, p, p, p, p, p, p, p, p, p, p, i64, p],
        "rc_grad_norm_workspace": [p, p, p, p],
        "rc_grad_norm": [p, p, p, p, p, i64, p],
        "rc_adamw_table": [p, p, p, p, p],
        "rc_adamw_step": [p, p, p, p, p, p, p],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32


def _outputs(out, present, what):
    """`out`'s lists in their places, None for those that the call does not have."""
    if out is None:
        return [None] * len(present)
    lists = [out] if sum(present) == 1 else out
    if sum(present) > 1 and (not isinstance(out, (tuple, list)) or len(out) != sum(present)):
        raise _rr.CollectiveError(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: out is not {sum(present)} lists of tensors")
    given = iter(lists)
    return [next(given) if p else None for p in present]


# ---------------------------------------------------------------- norm

def rms_norm(xs, weights, eps=1e-6, residuals=None, quantize=None, group=None, out=None, stream=None):
    """Root-mean-square norm of every row: s / sqrt(mean(s^2) + eps) * weight,
    with s = xs[r] or, given residuals, xs[r] + residuals[r] as rounded to the
    rows' type.  xs[r] is [tokens, width], weights[r] [width], of the rows' type
    or float32 (the same tensor for all ranks will do).  Returns ys; with
    quantize="e4m3" ys are float8_e4m3fn and scales [tokens, groups] follow (a
    scale for a row, or for each `group` of 32, 64, 128 or 256 elements), with
    residuals the sums follow: ys, (ys, scales), (ys, sums) or (ys, scales,
    sums), as `out` is given too.  In place: the sums may be the residuals, and
    ys the xs."""
    quantize = _choice(QUANTIZE, quantize, "rms_norm: quantize")
    ys, scales, sums = _outputs(out, (True, bool(quantize), residuals is not None), "rms_norm")
    return _call("rms_norm", stream, xs, weights, eps, residuals, quantize, group or 0, ys, scales, sums)


def rms_norm_grad(d_ys, sums, weights, eps=1e-6, d_sums=None, out=None, stream=None):
    """The gradients of rms_norm: (d_xs, d_weights).  sums are the rows that were
    normalised (xs without residuals), d_sums what comes back by the sums
    themselves; d_xs is the gradient of the residuals too.  d_weights[r] is summed
    over rank r's rows, of the weights' type.  d_xs may be d_ys or d_sums."""
    return _call("rms_norm_grad", stream, d_ys, sums, weights, eps, d_sums, out)


# ---------------------------------------------------------------- experts

def moe_layer(xs, weights, experts, gate_up, down, scales=None, gate_up_scales=None, down_scales=None, dtype=None,
              out=None, stream=None):
    """A mixture-of-experts layer for a few tokens (all ranks' tokens times top_k
    up to 2048; dispatch and combine take any number): ys[r][t] = the sum over k
    of weights[r][t, k] * down (silu(gate x) * (up x)) with the matrices of
    expert experts[r][t, k], as route gives them (-1: none).  xs[r] is [tokens,
    width]; rank d holds the weights of its experts, gate_up[d] [experts of a
    rank, 2 * inner, width] (gate above up) and down[d] [experts, width, inner],
    of the rows' type or, with 16-bit rows, float8_e4m3fn with gate_up_scales
    [experts, 2 * inner] and down_scales [experts, width], float32 factors of the
    rows.  8-bit rows (rms_norm's with a scale a row: scales [tokens, 1]) take
    8-bit weights, and give ys of `dtype` (bfloat16 unless said or as `out` has
    it).  The chosen experts' weights are read where they lie, once for every 64 to
    128 entries of an expert."""
    return _call("moe_layer", stream, xs, weights, experts, gate_up, down, scales, gate_up_scales, down_scales, dtype, out)


# ---------------------------------------------------------------- gradient norms and AdamW

def grad_norm(grads, over="rank", out=None, stream=None):
    """The 2-norm of each rank's gradients, grads[r] a map {parameter id: tensor}
    (None for a parameter without one): a float32 tensor of R on the GPU, summed
    in 64 bits.  over="all": every rank's is that of all ranks' gradients, for
    parameters sharded over the ranks."""
    if over not in ("rank", "all"):
        raise _rr.CollectiveError(_rr.RC_ERR_INVALID_ARGUMENT, f"grad_norm: over {over!r} is neither 'rank' nor 'all'")
    return _call("grad_norm", stream, grads, over == "all", out)


class AdamWState:
    """The ranks' parameters with their AdamW state, one map {parameter id:
    tensor} per rank each:
      params          float32, or 16 bits with a float32 copy in `master`;
      m, v            means of the gradients and of their squares: float32, or
                      with bits=8 float8_e4m3fn codes of m and of the root of v
                      with float32 scales of 256 elements each in m_scale, v_scale;
      step            int32, one number for each rank: the steps made, whichever
                      parameters had gradients in them.
    The tensors are updated in place by adamw_step, which goes by their addresses
    from here: copy into them to change them (others put into the maps are not
    seen); it refuses a state whose tensors have been given other memory.  A state
    made from saved tensors goes on where they were saved.  It has to live until a
    step on a stream that is not torch's own (a number, an ExternalStream) is done,
    and as long as a graph that holds a step is replayed; with torch's streams the
    tensors alone do."""

    __slots__ = ("bits", "params", "m", "v", "step", "master", "m_scale", "v_scale", "_table")

    def __init__(self, params, bits, m, v, step, master=None, m_scale=None, v_scale=None):
        self.bits, self.params, self.m, self.v, self.step = bits, params, m, v, step
        self.master, self.m_scale, self.v_scale = master, m_scale, v_scale
        self._table = _call("adamw_table", None, bits, params, master, m, v, m_scale, v_scale)


def adamw_state(params, bits=32):
    """A new state for params, one map {parameter id: tensor} per rank: means of
    zero, 32 or 8 bits each, and float32 copies of 16-bit parameters."""
    torch = _rr._torch()
    dtype = torch.float8_e4m3fn if bits == 8 else torch.float32

    def zeros():
        return [{k: torch.zeros(p.shape, dtype=dtype, device=p.device) for k, p in m.items()} for m in params]

    def scales():
        return [{k: torch.zeros(-(-p.numel() // 256), device=p.device) for k, p in m.items()} for m in params]

    master = [{k: p.detach().float() for k, p in m.items() if p.dtype != torch.float32} for m in params]
    device = next((p.device for m in params for p in m.values()), None)
    return AdamWState(params, bits, zeros(), zeros(), torch.zeros(len(params), dtype=torch.int32, device=device),
                      master=master, m_scale=scales() if bits == 8 else None, v_scale=scales() if bits == 8 else None)


def adamw_step(state, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, norms=None, max_norm=None,
               grad_scale=1.0, seed=0, out=None, stream=None):
    """One AdamW step of every parameter that has a gradient, grads[r] a map
    {parameter id: tensor} of the parameters' types or float32 (include/rc.h has
    the formulas).  norms are grad_norm's: a rank whose norm is not finite makes
    no step, and with max_norm larger gradients are scaled down to it, both
    decided on the GPU.  grad_scale: a factor of the gradients before all that.
    lr: a number, or a float32 tensor of one element on the GPU, for steps
    captured into a graph.  8-bit states are rounded by chance, as `seed`, the
    step and the element's place say: v's, and m's where it has no gradient and
    would stay.  In place, or into `out`, another state of the same parameters.
    Steps of one state run one after the other."""
    to = state if out is None else out
    _call("adamw_step", stream, state._table, state.step, to._table, to.step, grads, lr, betas[0], betas[1], eps,
          weight_decay, norms, 0.0 if max_norm is None else max_norm, grad_scale, seed)
    return to
