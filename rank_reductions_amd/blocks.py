"""Block operators: what stands around a mixture-of-experts block and behind a
gradient sync (whole-call form; include/rc.h, "Block operators").

    ys, sums = rr.rms_norm(xs, weights, residuals=hs)      # R tensors each
    codes, scales, sums = rr.rms_norm(xs, weights, residuals=hs, quantize="e4m3")
    d_xs, d_weights = rr.rms_norm_grad(d_ys, sums, weights, d_sums=d_hs)

Argument marshalling only, as of the row exchanges (rows.py): tensors are given
as one per rank, on the session's GPU; new ones are allocated, and kernels
enqueued, on `stream` (the current one if None), and the parts of one call may
share an allocation.
"""

import ctypes

import rank_reductions_amd as _rr
from rank_reductions_amd.rows import _call, _choice

__all__ = ["rms_norm", "rms_norm_grad"]

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


def declare(lib):
    """Argument types of the library's block operators."""
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name, args in {
        "rc_rms_norm": [p, p, p, p, p, p, p, p],
        "rc_rms_norm_grad_workspace": [p, p],
        "rc_rms_norm_grad": [p, p, p, p, p, p, p, p, i64, p],
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
