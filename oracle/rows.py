"""Row exchanges in 64 bits: expert routing, dispatch and combine, the sharded
embedding and its gradient, straight from their definitions, one token at a
time.  Inputs and outputs are NumPy arrays, one per rank.
"""

import numpy as np


def _scores(x, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max()
        if not np.isfinite(top):  # nothing but -inf, or a NaN or +inf: no score is a number
            return np.full_like(x, np.nan)
        e = np.exp(x - top)
        return e / e.sum()


def route_token(x, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_by="top2", renormalize=True,
                scale=1.0):
    """(weights, experts) of one token's logits x."""
    x = np.asarray(x, dtype=np.float64)
    s = _scores(x, score)
    c = s.copy()
    if bias is not None:
        c = c + np.asarray(bias, dtype=np.float64)
    c[(x == -np.inf) | np.isnan(c)] = -np.inf
    size = x.size // groups
    if groups > 1:
        best = []
        for g in range(groups):
            v = sorted(c[g * size:(g + 1) * size], reverse=True)
            best.append(v[0] + v[1] if group_by == "top2" and size > 1 else v[0])
        kept = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        for g in range(groups):
            if g not in kept:
                c[g * size:(g + 1) * size] = -np.inf
    order = sorted(range(x.size), key=lambda e: (-c[e], e))[:top_k]
    experts = [e if c[e] > -np.inf else -1 for e in order]
    w = np.array([s[e] if e >= 0 else 0.0 for e in experts])
    if renormalize:
        total = w.sum()
        w = w / total if total > 0 else np.zeros_like(w)
    return scale * w, np.array(experts, dtype=np.int32)


def route(logits, top_k, **kw):
    weights, experts = [], []
    for l in logits:
        rows = [route_token(x, top_k, **kw) for x in l]
        weights.append(np.array([r[0] for r in rows]).reshape(-1, top_k))
        experts.append(np.array([r[1] for r in rows], dtype=np.int32).reshape(-1, top_k))
    return weights, experts


def route_grad_token(x, experts, d_weights, score="softmax", renormalize=True, scale=1.0):
    """d_logits of one token: the chain of derivatives, weights by scores by logits."""
    x = np.asarray(x, dtype=np.float64)
    dx = np.zeros_like(x)
    slots = [k for k, e in enumerate(experts) if 0 <= e < x.size]
    if not slots:
        return dx
    s = _scores(x, score)
    at = [experts[k] for k in slots]
    p = s[at]
    g = scale * np.array([d_weights[k] for k in slots], dtype=np.float64)
    if renormalize:
        # w = p / sum(p): a softmax's common factor cancels, so it has a part
        # in the chosen logits only
        total = p.sum()
        if not total > 0:
            return dx
        q = p / total
        part = q * (g - (g * q).sum())
        if score == "sigmoid":
            part = part * (1.0 - p)
        np.add.at(dx, at, part)
        return dx
    if score == "sigmoid":
        np.add.at(dx, at, g * p * (1.0 - p))
        return dx
    np.add.at(dx, at, g * p)
    return dx - s * (g * p).sum()


def route_grad(logits, experts, d_weights, **kw):
    return [np.array([route_grad_token(x, e, d, **kw) for x, e, d in zip(*rank)]).reshape(np.shape(rank[0]))
            for rank in zip(logits, experts, d_weights)]


def dispatch_plan(experts, num_experts, capacity):
    """(slots, offsets, counts): each rank's rows by expert, source rank, token, k."""
    R = len(experts)
    per = num_experts // R
    slots = [np.full(e.shape, -1, dtype=np.int32) for e in experts]
    offsets, counts = [], []
    for d in range(R):
        row, starts, held = 0, [], []
        for e in range(d * per, (d + 1) * per):
            starts.append(min(row, capacity[d]))
            first = row
            for r in range(R):
                for t, k in zip(*np.nonzero(experts[r] == e)):
                    if row < capacity[d]:
                        slots[r][t, k] = row
                    row += 1
            held.append(row - first)
        offsets.append(np.array(starts + [min(row, capacity[d])], dtype=np.int32))
        counts.append(np.array(held, dtype=np.int32))
    return slots, offsets, counts


def places(experts, slots, num_experts):
    """(source rank, token, k, destination rank, slot) of every placed entry."""
    per = num_experts // len(experts)
    for r, (e, s) in enumerate(zip(experts, slots)):
        for t, k in zip(*np.nonzero(s >= 0)):
            yield r, t, k, int(e[t, k]) // per, int(s[t, k])


def dispatch(xs, experts, slots, num_experts, rows):
    """Writes the placed rows into copies of `rows`."""
    out = [x.copy() for x in rows]
    for r, t, _, d, s in places(experts, slots, num_experts):
        out[d][s] = xs[r][t]
    return out


def combine(rows, experts, slots, num_experts, weights=None):
    """(sums, sums of the absolute values): the second scales error bounds."""
    width = rows[0].shape[1]
    out = [np.zeros((e.shape[0], width)) for e in experts]
    size = [np.zeros((e.shape[0], width)) for e in experts]
    for r, t, k, d, s in places(experts, slots, num_experts):
        v = rows[d][s].astype(np.float64) * (1.0 if weights is None else float(weights[r][t, k]))
        out[r][t] += v
        size[r][t] += np.abs(v)
    return out, size


def combine_grad(d_outs, rows, experts, slots, num_experts, weights, d_rows):
    """(d_rows, d_weights, sums of the products' absolute values); d_rows into copies of `d_rows`."""
    dr = [x.astype(np.float64) for x in d_rows]
    dw = [np.zeros(e.shape) for e in experts]
    size = [np.zeros(e.shape) for e in experts]
    for r, t, k, d, s in places(experts, slots, num_experts):
        dy, x = d_outs[r][t].astype(np.float64), rows[d][s].astype(np.float64)
        dr[d][s] = float(weights[r][t, k]) * dy
        dw[r][t, k] = (dy * x).sum()
        size[r][t, k] = np.abs(dy * x).sum()
    return dr, dw, size


def shard_bounds(vocab, num_ranks):
    s = -(-vocab // num_ranks)
    return [(min(c * s, vocab), min((c + 1) * s, vocab)) for c in range(num_ranks)]


def embedding(ids, table, scale=1.0):
    """Rows of the whole table; zeros for ids outside it."""
    out = []
    for i in ids:
        y = np.zeros((i.size, table.shape[1]))
        for t, v in enumerate(i):
            if 0 <= v < table.shape[0]:
                y[t] = scale * table[v].astype(np.float64)
        out.append(y)
    return out


PIECE, RUN = 64, 16


def embedding_grad(ids, d_outs, vocab, scale=1.0):
    """(gradient of the whole table, sums of absolute values, tokens of each id)."""
    width = d_outs[0].shape[1]
    out, size, count = np.zeros((vocab, width)), np.zeros((vocab, width)), np.zeros(vocab, dtype=np.int64)
    for i, d in zip(ids, d_outs):
        for t, v in enumerate(i):
            if 0 <= v < vocab:
                x = scale * d[t].astype(np.float64)
                out[v] += x
                size[v] += np.abs(x)
                count[v] += 1
    return out, size, count


def embedding_grad_ordered(ids, d_outs, vocab, scale=1.0, old=None):
    """The same in float32, in the documented order: pieces of 64 tokens summed
    from zero, runs of 16 pieces likewise, the runs added in order; then the
    scale, then the old value.  Rows in float32 as they are before the last
    rounding; `old` (or zeros) where no token names the row."""
    width = d_outs[0].shape[1]
    rows = {}
    for i, d in zip(ids, d_outs):
        for t, v in enumerate(i):
            if 0 <= v < vocab:
                rows.setdefault(int(v), []).append(d[t].astype(np.float32))

    def add_up(parts):
        total = np.zeros(width, dtype=np.float32)
        for p in parts:
            total = total + p
        return total

    def in_parts(parts, size):
        return [add_up(parts[i:i + size]) for i in range(0, len(parts), size)]

    out = np.zeros((vocab, width), dtype=np.float32) if old is None else old.astype(np.float32)
    for v, parts in rows.items():
        if len(parts) > PIECE:
            total = add_up(in_parts(in_parts(parts, PIECE), RUN))
        else:
            total = add_up(parts)
        total = total * np.float32(scale)
        out[v] = total if old is None else total + out[v]
    return out
