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

Argument marshalling only: the kernels run in librankred.so.  Tensors are
given as one per rank, on the session's GPU; new ones are allocated, and
kernels enqueued, on `stream` (the current one if None).
"""

import contextlib
import ctypes

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
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i32


# ---------------------------------------------------------------- checks

def _fail(code, message):
    raise _rr.CollectiveError(code, message)


def _row_type(t, what):
    torch = _rr._torch()
    code = {torch.float32: _rr.RC_F32, torch.float16: RC_F16, torch.bfloat16: RC_BF16}.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}; float32, float16 and bfloat16 are supported")
    return code


def _session(what, xs):
    """Checks that the list has one tensor per rank of the open session, on
    its GPU.  Returns the rank count and the device."""
    n, d = ctypes.c_int(), ctypes.c_int()
    _rr.check(_rr.library().rc_session_info(ctypes.byref(n), ctypes.byref(d)))
    if len(xs) != n.value:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: {len(xs)} tensors for {n.value} ranks")
    device = xs[0].device
    if device.type == "cuda" and d.value >= 0 and device.index != d.value:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: tensors on {device}, the session on GPU {d.value}")
    return n.value, device


def _same(ts, n, shape_of, dtype, device, what):
    """Every rank's tensor has its shape, one dtype, one device, and is dense."""
    if len(ts) != n:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: {len(ts)} tensors for {n} ranks")
    for r, t in enumerate(ts):
        if t is None:
            _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: no tensor for rank {r}")
        if t.dtype != dtype:
            _fail(_rr.RC_ERR_DTYPE_MISMATCH, f"{what}: rank {r} has dtype {t.dtype}, expected {dtype}")
        if tuple(t.shape) != shape_of(r):
            _fail(_rr.RC_ERR_SHAPE_MISMATCH, f"{what}: rank {r} has shape {tuple(t.shape)}, expected {shape_of(r)}")
        if t.device != device:
            _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: rank {r} on {t.device}, others on {device}")
        if not t.is_contiguous():
            _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: rank {r} is not contiguous")


def _matrix(ts, what):
    for r, t in enumerate(ts):
        if t.dim() != 2:
            _fail(_rr.RC_ERR_SHAPE_MISMATCH, f"{what}: rank {r} has {t.dim()} dimensions, expected [tokens, width]")


def _ptrs(ts):
    # Sequences of addresses; all were checked to be dense.
    if not ts[0].is_cuda:
        raise ValueError("tensors must be on a CUDA (HIP) device")
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _counts(values):
    return (ctypes.c_int64 * len(values))(*values)


def _on(stream):
    """The context that allocates on `stream`."""
    if stream is None:
        return contextlib.nullcontext()
    torch = _rr._torch()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _addr(array):
    return ctypes.addressof(array)


def _choice(table, value, what):
    if value not in table:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what} {value!r} is none of {', '.join(table)}")
    return table[value]


# ---------------------------------------------------------------- routing

def _route_desc(t, top_k, score, bias, groups, top_groups, group_by, renormalize, scale, what):
    d = RcRouteDesc()
    d.struct_size = ctypes.sizeof(RcRouteDesc)
    d.dtype = _row_type(t, what)
    d.num_experts = t.shape[1]
    d.top_k = top_k
    d.score = _choice(SCORES, score, f"{what}: score")
    d.num_groups = groups
    d.top_groups = top_groups
    d.group_by = _choice(GROUP_BY, group_by, f"{what}: group_by")
    d.renormalize = 1 if renormalize else 0
    d.scale = scale
    d.bias = bias.data_ptr() if bias is not None else None
    return d


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
    torch = _rr._torch()
    what = "route"
    n, dev = _session(what, logits)
    _matrix(logits, what)
    E = logits[0].shape[1]
    tokens = [t.shape[0] for t in logits]
    _same(logits, n, lambda r: (tokens[r], E), logits[0].dtype, dev, what)
    if bias is not None:
        _same([bias], 1, lambda r: (E,), torch.float32, dev, "route bias")
    d = _route_desc(logits[0], top_k, score, bias, groups, top_groups, group_by, renormalize, scale, what)
    if out is None:
        with _on(stream):
            out = ([torch.empty(t, top_k, dtype=torch.float32, device=dev) for t in tokens],
                   [torch.empty(t, top_k, dtype=torch.int32, device=dev) for t in tokens])
    weights, experts = out
    _same(weights, n, lambda r: (tokens[r], top_k), torch.float32, dev, "route weights")
    _same(experts, n, lambda r: (tokens[r], top_k), torch.int32, dev, "route experts")
    _rr.check(_rr.library().rc_route(ctypes.byref(d), _counts(tokens), _ptrs(logits), _ptrs(weights),
                                     _ptrs(experts), _rr._stream(stream, logits[0])))
    return weights, experts


def route_grad(logits, experts, d_weights, score="softmax", renormalize=True, scale=1.0, out=None, stream=None):
    """The gradient of route's weights for the experts it chose: d_logits, R
    tensors like logits."""
    torch = _rr._torch()
    what = "route_grad"
    n, dev = _session(what, logits)
    _matrix(logits, what)
    E = logits[0].shape[1]
    tokens = [t.shape[0] for t in logits]
    _same(logits, n, lambda r: (tokens[r], E), logits[0].dtype, dev, what)
    if len(experts) != n:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what} experts: {len(experts)} tensors for {n} ranks")
    _matrix(experts, what + " experts")
    K = experts[0].shape[1]
    _same(experts, n, lambda r: (tokens[r], K), torch.int32, dev, what + " experts")
    _same(d_weights, n, lambda r: (tokens[r], K), torch.float32, dev, what + " d_weights")
    d = _route_desc(logits[0], K, score, None, 1, 1, "max", renormalize, scale, what)
    if out is None:
        with _on(stream):
            out = [torch.empty_like(t) for t in logits]
    _same(out, n, lambda r: (tokens[r], E), logits[0].dtype, dev, what + " output")
    _rr.check(_rr.library().rc_route_grad(ctypes.byref(d), _counts(tokens), _ptrs(logits), _ptrs(experts),
                                          _ptrs(d_weights), _ptrs(out), _rr._stream(stream, logits[0])))
    return out


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

    def __init__(self, experts, slots, offsets, counts, num_experts, capacity):
        self.experts, self.slots, self.offsets, self.counts = experts, slots, offsets, counts
        self.num_experts, self.capacity = num_experts, capacity
        self.tokens = [t.shape[0] for t in experts]
        self.top_k = experts[0].shape[1]


def _exchange_desc(plan, dtype, width):
    """The descriptor and the arrays that it points to (kept with it)."""
    d = RcExchangeDesc()
    d.struct_size = ctypes.sizeof(RcExchangeDesc)
    d.dtype = dtype
    d.num_experts = plan.num_experts
    d.top_k = plan.top_k
    d.width = width
    d.held = (_counts(plan.tokens), _counts(plan.capacity), _ptrs(plan.experts), _ptrs(plan.slots))
    d.tokens, d.capacity, d.experts, d.slots = map(_addr, d.held)
    return d


def dispatch_plan(experts, num_experts, capacity=None, stream=None):
    """Places every token on the ranks of its experts (experts[r]: [tokens,
    top_k] int32, -1 for none; rank d holds num_experts / R consecutive
    experts).  Each rank's rows are ordered by expert, then source rank, token
    and k.  capacity: rows per rank, one number or one per rank; entries past
    it have no place (slot -1).  None makes room for all."""
    torch = _rr._torch()
    what = "dispatch_plan"
    n, dev = _session(what, experts)
    _matrix(experts, what)
    K = experts[0].shape[1]
    tokens = [t.shape[0] for t in experts]
    _same(experts, n, lambda r: (tokens[r], K), torch.int32, dev, what)
    if num_experts < 1 or num_experts % n:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: {num_experts} experts over {n} ranks")
    if capacity is None:
        capacity = sum(tokens) * K
    capacity = [int(capacity)] * n if not isinstance(capacity, (list, tuple)) else [int(c) for c in capacity]
    if len(capacity) != n:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: {len(capacity)} capacities for {n} ranks")
    per = num_experts // n
    with _on(stream):
        sizes = [t * K for t in tokens] + [per + 1] * n + [per] * n
        parts = torch.empty(sum(sizes), dtype=torch.int32, device=dev).split(sizes)
        plan = DispatchPlan(list(experts), [p.view(t, K) for p, t in zip(parts, tokens)], list(parts[n:2 * n]),
                            list(parts[2 * n:]), num_experts, capacity)
        d = _exchange_desc(plan, _rr.RC_F32, 1)
        size = ctypes.c_int64()
        _rr.check(_rr.library().rc_dispatch_plan_workspace(ctypes.byref(d), ctypes.byref(size)))
        work = torch.empty(size.value, dtype=torch.uint8, device=dev)
    _rr.check(_rr.library().rc_dispatch_plan(ctypes.byref(d), _ptrs(plan.offsets), _ptrs(plan.counts),
                                             work.data_ptr() or None, size.value, _rr._stream(stream, experts[0])))
    return plan


def _check_plan(plan, n, dev, what):
    _same(plan.experts, n, lambda r: (plan.tokens[r], plan.top_k), _rr._torch().int32, dev, what + " experts")
    _same(plan.slots, n, lambda r: (plan.tokens[r], plan.top_k), _rr._torch().int32, dev, what + " slots")


def dispatch(xs, plan, out=None, stream=None):
    """Each token's row to its places: out[d][slot] = xs[r][token].  Returns
    one [capacity, width] tensor per rank; rows behind offsets[d][-1] are not
    written (zeros in a tensor allocated here)."""
    torch = _rr._torch()
    what = "dispatch"
    n, dev = _session(what, xs)
    _matrix(xs, what)
    D = xs[0].shape[1]
    _same(xs, n, lambda r: (plan.tokens[r], D), xs[0].dtype, dev, what)
    _check_plan(plan, n, dev, what)
    if out is None:
        with _on(stream):
            out = [torch.zeros(c, D, dtype=xs[0].dtype, device=dev) for c in plan.capacity]
    _same(out, n, lambda r: (plan.capacity[r], D), xs[0].dtype, dev, what + " output")
    d = _exchange_desc(plan, _row_type(xs[0], what), D)
    _rr.check(_rr.library().rc_dispatch(ctypes.byref(d), _ptrs(xs), _ptrs(out), _rr._stream(stream, xs[0])))
    return out


def combine(rows, plan, weights=None, out=None, stream=None):
    """Each token's rows back: out[r][token] = sum over k of weights[r][token,
    k] * rows[d][slot], in order of k.  Without weights all count one, which
    is dispatch's gradient."""
    torch = _rr._torch()
    what = "combine"
    n, dev = _session(what, rows)
    _matrix(rows, what)
    D = rows[0].shape[1]
    _same(rows, n, lambda r: (plan.capacity[r], D), rows[0].dtype, dev, what)
    _check_plan(plan, n, dev, what)
    if weights is not None:
        _same(weights, n, lambda r: (plan.tokens[r], plan.top_k), torch.float32, dev, what + " weights")
    if out is None:
        with _on(stream):
            out = [torch.empty(t, D, dtype=rows[0].dtype, device=dev) for t in plan.tokens]
    _same(out, n, lambda r: (plan.tokens[r], D), rows[0].dtype, dev, what + " output")
    d = _exchange_desc(plan, _row_type(rows[0], what), D)
    _rr.check(_rr.library().rc_combine(ctypes.byref(d), _ptrs(rows), None if weights is None else _ptrs(weights),
                                       _ptrs(out), _rr._stream(stream, rows[0])))
    return out


def combine_grad(d_outs, rows, plan, weights, out=None, stream=None):
    """The gradients of combine: (d_rows, d_weights).  Rows of d_rows that no
    token has are not written (zeros in a tensor allocated here)."""
    torch = _rr._torch()
    what = "combine_grad"
    n, dev = _session(what, d_outs)
    _matrix(d_outs, what)
    D, dt = d_outs[0].shape[1], d_outs[0].dtype
    _same(d_outs, n, lambda r: (plan.tokens[r], D), dt, dev, what)
    _same(rows, n, lambda r: (plan.capacity[r], D), dt, dev, what + " rows")
    _check_plan(plan, n, dev, what)
    _same(weights, n, lambda r: (plan.tokens[r], plan.top_k), torch.float32, dev, what + " weights")
    if out is None:
        with _on(stream):
            out = ([torch.zeros(c, D, dtype=dt, device=dev) for c in plan.capacity],
                   [torch.empty_like(w) for w in weights])
    d_rows, d_weights = out
    _same(d_rows, n, lambda r: (plan.capacity[r], D), dt, dev, what + " d_rows")
    _same(d_weights, n, lambda r: (plan.tokens[r], plan.top_k), torch.float32, dev, what + " d_weights")
    d = _exchange_desc(plan, _row_type(d_outs[0], what), D)
    _rr.check(_rr.library().rc_combine_grad(ctypes.byref(d), _ptrs(d_outs), _ptrs(rows), _ptrs(weights),
                                            _ptrs(d_rows), _ptrs(d_weights), _rr._stream(stream, d_outs[0])))
    return d_rows, d_weights


# ---------------------------------------------------------------- embedding

def shard_rows(vocab, num_ranks):
    """Rows of a vocabulary table on each rank: segments of ceil(vocab / R)."""
    s = -(-vocab // num_ranks)
    return [max(0, min((c + 1) * s, vocab) - c * s) for c in range(num_ranks)]


def _check_ids(ids, n, dev, what):
    torch = _rr._torch()
    for r, t in enumerate(ids):
        if t.dim() != 1:
            _fail(_rr.RC_ERR_SHAPE_MISMATCH, f"{what}: rank {r} has {t.dim()} dimensions, expected [tokens]")
    if ids[0].dtype not in (torch.int32, torch.int64):
        raise TypeError(f"{what}: unsupported dtype {ids[0].dtype}; int32 and int64 are supported")
    tokens = [t.shape[0] for t in ids]
    _same(ids, n, lambda r: (tokens[r],), ids[0].dtype, dev, what)
    return tokens


def _embedding_desc(ids, tokens, dtype, grad_dtype, accumulate, scale, vocab, width):
    d = RcEmbeddingDesc()
    d.struct_size = ctypes.sizeof(RcEmbeddingDesc)
    d.dtype, d.grad_dtype = dtype, grad_dtype
    d.id_dtype = RC_I64 if ids[0].dtype == _rr._torch().int64 else _rr.RC_I32
    d.accumulate = 1 if accumulate else 0
    d.scale = scale
    d.vocab, d.width = vocab, width
    d.held = (_counts(tokens), _ptrs(ids))
    d.tokens, d.ids = map(_addr, d.held)
    return d


def embedding(ids, tables, scale=1.0, out=None, stream=None):
    """scale * table[id] for every token: ids[r] is [tokens] (int32 or int64),
    tables[c] rank c's rows of the vocabulary (shard_rows(vocab, R) of them).
    An id outside the vocabulary gives zeros.  Returns [tokens, width] for
    each rank."""
    torch = _rr._torch()
    what = "embedding"
    n, dev = _session(what, ids)
    tokens = _check_ids(ids, n, dev, what)
    if len(tables) != n:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: {len(tables)} tables for {n} ranks")
    _matrix(tables, what)
    D, vocab = tables[0].shape[1], sum(t.shape[0] for t in tables)
    rows = shard_rows(vocab, n)
    _same(tables, n, lambda r: (rows[r], D), tables[0].dtype, dev, what + " tables")
    code = _row_type(tables[0], what)
    if out is None:
        with _on(stream):
            out = [torch.empty(t, D, dtype=tables[0].dtype, device=dev) for t in tokens]
    _same(out, n, lambda r: (tokens[r], D), tables[0].dtype, dev, what + " output")
    d = _embedding_desc(ids, tokens, code, code, False, scale, vocab, D)
    _rr.check(_rr.library().rc_embedding(ctypes.byref(d), _ptrs(tables), _ptrs(out), _rr._stream(stream, ids[0])))
    return out


def embedding_grad(ids, d_outs, vocab, scale=1.0, dtype=None, out=None, accumulate=False, stream=None):
    """The gradient of embedding's table, summed over all ranks' tokens in
    order of rank and token, one tensor of rows per rank as in embedding; of
    d_outs' type, or float32 (`dtype`, or that of `out`).  With accumulate the
    sums are added to `out`."""
    torch = _rr._torch()
    what = "embedding_grad"
    n, dev = _session(what, ids)
    tokens = _check_ids(ids, n, dev, what)
    if len(d_outs) != n:
        _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: {len(d_outs)} gradients for {n} ranks")
    _matrix(d_outs, what)
    D = d_outs[0].shape[1]
    _same(d_outs, n, lambda r: (tokens[r], D), d_outs[0].dtype, dev, what)
    rows = shard_rows(vocab, n)
    if out is None:
        if accumulate:
            _fail(_rr.RC_ERR_INVALID_ARGUMENT, f"{what}: accumulate needs the tensors to add to")
        with _on(stream):
            out = [torch.empty(v, D, dtype=dtype or d_outs[0].dtype, device=dev) for v in rows]
    _same(out, n, lambda r: (rows[r], D), dtype or out[0].dtype, dev, what + " output")
    d = _embedding_desc(ids, tokens, _row_type(d_outs[0], what), _row_type(out[0], what), accumulate, scale, vocab, D)
    size = ctypes.c_int64()
    _rr.check(_rr.library().rc_embedding_grad_workspace(ctypes.byref(d), ctypes.byref(size)))
    with _on(stream):
        work = torch.empty(size.value, dtype=torch.uint8, device=dev)
    _rr.check(_rr.library().rc_embedding_grad(ctypes.byref(d), _ptrs(d_outs), _ptrs(out), work.data_ptr() or None,
                                              size.value, _rr._stream(stream, ids[0])))
    return out
