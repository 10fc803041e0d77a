"""Row exchanges: operators that move rows between the ranks by an index
computed on the GPU (whole-call form; include/rc.h, "Row exchanges").

Expert parallelism - `route` chooses each token's experts, `dispatch_plan`
places the tokens on the experts' ranks, `dispatch` and `combine` move the rows
there and back:

    weights, experts = rr.route(logits, top_k=8)          # R tensors each
    plan = rr.dispatch_plan(experts, num_experts=64)
    rows = rr.dispatch(xs, plan)                          # rows[d][:plan.offsets[d][-1]]
    ys = rr.combine(results, plan, weights)
    d_results, d_weights = rr.combine_grad(d_ys, results, plan, weights)
    d_xs = rr.combine(d_rows, plan)                       # dispatch's gradient
    d_logits = rr.route_grad(logits, experts, d_weights)

A vocabulary table sharded over the ranks - `embedding` looks rows up, and
`embedding_grad` sums the gradient over the tokens of all ranks.

Argument marshalling only, most of it in the native module _rows: the kernels
run in librankred.so.  Tensors are given as one per rank, on the session's
GPU; new ones are allocated, and kernels enqueued, on `stream` (a stream of that
GPU; the current one if None).  As with torch's functions, tensors that belong
to another stream have to live until `stream` is done with them
(Tensor.record_stream).

New tensors of one call are parts of one allocation while all ranks' together
are at most 16 MiB, and a plan's slots, offsets and counts always are: like the
parts that torch.split gives, each keeps the whole alive, is saved with the
whole, and must not be grown in place (resize_), which would run into the next.
Give `out` where that matters.
"""

import ctypes
import importlib
import threading
from pathlib import Path

import rank_reductions_amd as _rr

__all__ = ["route", "route_grad", "DispatchPlan", "dispatch_plan", "dispatch", "combine", "combine_grad",
           "embedding", "embedding_grad"]

RC_F16, RC_BF16, RC_I64 = 2, 3, 4
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_BY = {"max": 0, "top2": 1}


class RcRouteDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_by", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("bias", ctypes.c_void_p),
        ("session", ctypes.c_int64),
    ]


class RcExchangeDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("width", ctypes.c_int64),
        ("tokens", ctypes.c_void_p),
        ("capacity", ctypes.c_void_p),
        ("experts", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("session", ctypes.c_int64),
    ]


class RcEmbeddingDesc(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("dtype", ctypes.c_int32),
        ("id_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("vocab", ctypes.c_int64),
        ("width", ctypes.c_int64),
        ("tokens", ctypes.c_void_p),
        ("ids", ctypes.c_void_p),
        ("session", ctypes.c_int64),
    ]


def declare(lib):
    """Argument types of the library's row-exchange entry points."""
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name, args in {
        "rc_route": [p, p, p, p, p, p],
        "rc_route_grad": [p, p, p, p, p, p, p],
        "rc_dispatch_plan_workspace": [p, p],
        "rc_dispatch_plan": [p, p, p, p, i64, p],
        "rc_dispatch": [p, p, p, p],
        "rc_combine": [p, p, p, p, p],
        "rc_combine_grad": [p, p, p, p, p, p, p],
        "rc_embedding": [p, p, p, p],
        "rc_embedding_grad_workspace": [p, p],
        "rc_embedding_grad": [p, p, p, p, i64, p],
        "rc_session_info": [p, p],
        "rc_session_id": [p],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32


# ---------------------------------------------------------------- the native module

_native_module = None
_native_lock = threading.Lock()


def _native():
    """The module _rows, loading it and the library on first use; raises if
    they are not built (no fallback exists)."""
    global _native_module
    if _native_module is not None:
        return _native_module
    with _native_lock:
        if _native_module is None:
            _rr._torch()
            _rr.library()
            path = Path(__file__).resolve().with_name("_rows.so")
            if not path.exists():
                raise RuntimeError(f"{path} is not built: run `python -m rank_reductions_amd.build` "
                                   "(no fallback implementation exists)")
            module = importlib.import_module("rank_reductions_amd._rows")
            module.set_error(_rr.CollectiveError)
            _native_module = module
    return _native_module


def _on(stream, what):
    """The context that makes `stream`, one of the session's GPU, current."""
    torch = _rr._torch()
    device = (_native_module or _native()).device()
    index = device if device >= 0 else None  # None: the current one
    if not hasattr(stream, "cuda_stream"):
        return torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=index))
    if index is not None and stream.device.index != index:
        raise _rr.CollectiveError(_rr.RC_ERR_INVALID_ARGUMENT,
                                  f"{what}: stream of {stream.device}, the session is on GPU {index}")
    return torch.cuda.stream(stream)


def _call(name, stream, *args):
    fn = getattr(_native_module or _native(), name)
    if stream is None:
        return fn(*args)
    with _on(stream, name):
        return fn(*args)


def _choice(table, value, what):
    code = table.get(value)
    if code is None:
        raise _rr.CollectiveError(_rr.RC_ERR_INVALID_ARGUMENT, f"{what} {value!r} is none of {', '.join(table)}")
    return code


# ---------------------------------------------------------------- routing

def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_by="top2", renormalize=True,
          scale=1.0, out=None, stream=None):
    """Chooses top_k experts for every token: logits[r] is [tokens, experts].
    Scores are the softmax or sigmoid of the logits; `bias` (float32
    [experts]) is added for the choice only; with groups > 1 only experts of
    the top_groups best groups are chosen (a group's score: its largest score,
    or with "top2" the sum of its two largest).  Returns (weights, experts),
    R tensors [tokens, top_k] each, float32 and int32: the chosen scores,
    divided by their sum with renormalize, times scale.  An expert with a
    logit of -inf is never chosen; slots left over hold expert -1, weight 0."""
    return _call("route", stream, logits, top_k, _choice(SCORES, score, "route: score"), bias, groups, top_groups,
                 _choice(GROUP_BY, group_by, "route: group_by"), renormalize, scale, out)


def route_grad(logits, experts, d_weights, score="softmax", renormalize=True, scale=1.0, out=None, stream=None):
    """The gradient of route's weights for the experts it chose: d_logits, R
    tensors like logits."""
    return _call("route_grad", stream, logits, experts, d_weights, _choice(SCORES, score, "route_grad: score"),
                 renormalize, scale, out)


# ---------------------------------------------------------------- dispatch and combine

class DispatchPlan:
    """Where each token's row goes (dispatch_plan):
      experts[r], slots[r]  [tokens, top_k]: the expert, and the row in its
                            rank's buffer or -1;
      offsets[d]            [experts of rank d + 1]: the first row of each of
                            rank d's experts, then the end;
      counts[d]             [experts of rank d]: entries that chose each
                            expert, also those past the capacity;
      capacity[d]           rows that rank d's buffer holds."""

    __slots__ = ("experts", "slots", "offsets", "counts", "num_experts", "capacity")

    def __init__(self, experts, slots, offsets, counts, num_experts, capacity):
        self.experts, self.slots, self.offsets, self.counts = experts, slots, offsets, counts
        self.num_experts, self.capacity = num_experts, capacity


def dispatch_plan(experts, num_experts, capacity=None, stream=None):
    """Places every token on the ranks of its experts (experts[r]: [tokens,
    top_k] int32, -1 for none; rank d holds num_experts / R consecutive
    experts).  Each rank's rows are ordered by expert, then source rank, token
    and k.  capacity: rows per rank, one number or one per rank; entries past
    it have no place (slot -1).  None makes room for all entries on every rank:
    R times the rows that are there, which dispatch and combine_grad hold, and
    clear, where they allocate.  Give a capacity, or `out`, for large batches."""
    slots, offsets, counts, capacity = _call("dispatch_plan", stream, experts, num_experts, capacity)
    return DispatchPlan(experts, slots, offsets, counts, num_experts, capacity)


def dispatch(xs, plan, out=None, stream=None):
    """Each token's row to its places: out[d][slot] = xs[r][token].  Returns
    one [capacity, width] tensor per rank; rows behind offsets[d][-1] are not
    written (zeros in a tensor allocated here)."""
    return _call("dispatch", stream, xs, plan.experts, plan.slots, plan.capacity, plan.num_experts, out)


def combine(rows, plan, weights=None, out=None, stream=None):
    """Each token's rows back: out[r][token] = sum over k of weights[r][token,
    k] * rows[d][slot], in order of k.  Without weights all count one, which
    is dispatch's gradient."""
    return _call("combine", stream, rows, plan.experts, plan.slots, plan.capacity, plan.num_experts, weights, out)


def combine_grad(d_outs, rows, plan, weights, out=None, stream=None):
    """The gradients of combine: (d_rows, d_weights).  Rows of d_rows that no
    token has are not written (zeros in a tensor allocated here)."""
    return _call("combine_grad", stream, d_outs, rows, plan.experts, plan.slots, plan.capacity, plan.num_experts,
                 weights, out)


# ---------------------------------------------------------------- embedding

def shard_rows(vocab, num_ranks):
    """Rows of a vocabulary table on each rank: segments of ceil(vocab / R)."""
    s = -(-vocab // num_ranks)
    return [max(0, min((c + 1) * s, vocab) - c * s) for c in range(num_ranks)]


def embedding(ids, tables, scale=1.0, out=None, stream=None):
    """scale * table[id] for every token: ids[r] is [tokens] (int32 or int64),
    tables[c] rank c's rows of the vocabulary (shard_rows(vocab, R) of them).
    An id outside the vocabulary gives zeros.  Returns [tokens, width] for
    each rank."""
    return _call("embedding", stream, ids, tables, scale, out)


def embedding_grad(ids, d_outs, vocab, scale=1.0, dtype=None, out=None, accumulate=False, stream=None):
    """The gradient of embedding's table, summed over all ranks' tokens in
    order of rank and token, one tensor of rows per rank as in embedding; of
    d_outs' type, or float32 (`dtype`, or that of `out`).  With accumulate the
    sums are added to `out`."""
    return _call("embedding_grad", stream, ids, d_outs, vocab, scale, dtype, out, accumulate)
