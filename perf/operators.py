"""The row-exchange operators' timed cases: expert routing, dispatch and
combine, the sharded embedding lookup and its gradient, each with its plain
form in elementary torch operations.

`own` selects the framework's kernels instead of the plain forms.  R logical
ranks hold their tokens in R tensors; experts and vocabulary rows are split
over the same ranks in order.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one decoding step of 64 sequences spread over 8 ranks: many experts in groups, sigmoid scores, balance bias
        dict(name="route_decode", kind="route", grad=False, ranks=8, tokens=8, ragged=False, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, group_by="top2", renormalize=True, scale=2.5,
             type="f32", padding=0.0),
        # a prompt batch of uneven lengths: softmax scores in 16 bits, where equal logits are common
        dict(name="route_prompt", kind="route", grad=False, ranks=8, tokens=4099, ragged=True, experts=128, top_k=8,
             score="softmax", bias=False, groups=1, top_groups=1, group_by="max", renormalize=True, scale=1.0,
             type="bf16", padding=0.02),
        # a training step's router over 131072 tokens, forward and backward
        dict(name="route_train", kind="route", grad=True, ranks=8, tokens=16384, ragged=False, experts=256, top_k=8,
             score="sigmoid", bias=True, groups=8, top_groups=4, group_by="top2", renormalize=True, scale=2.5,
             type="f32", padding=0.01),
        # one decoding step's tokens to their experts' ranks
        dict(name="dispatch_decode", kind="dispatch", ranks=8, tokens=8, ragged=False, experts=64, top_k=8,
             width=4096, type="bf16", room=8.0, padding=0.0),
        # an uneven prompt batch, 32-bit rows of an odd width, some tokens of padding, experts that overflow
        dict(name="dispatch_prompt", kind="dispatch", ranks=4, tokens=2049, ragged=True, experts=60, top_k=4,
             width=1001, type="f32", room=1.0, padding=0.05),
        # a training step's tokens, rows of the transformer's hidden size
        dict(name="dispatch_train", kind="dispatch", ranks=8, tokens=2048, ragged=False, experts=64, top_k=8,
             width=4096, type="bf16", room=2.0, padding=0.0),
        # the experts' results of one decoding step back to their tokens
        dict(name="combine_decode", kind="combine", grad=False, ranks=8, tokens=8, ragged=False, experts=64, top_k=8,
             width=4096, type="bf16", room=8.0, padding=0.0),
        # a training step's results back, and their gradients
        dict(name="combine_train", kind="combine", grad=True, ranks=8, tokens=2048, ragged=False, experts=64, top_k=8,
             width=4096, type="bf16", room=2.0, padding=0.0),
        # the tokens of one decoding step
        dict(name="embedding_decode", kind="embedding", ranks=8, tokens=8, ragged=False, vocab=32000, width=4096,
             type="bf16", ids="i32", scale=1.0, padding=0.0),
        # a training step's tokens, scaled by the square root of the width
        dict(name="embedding_train", kind="embedding", ranks=8, tokens=8192, ragged=False, vocab=32000, width=4096,
             type="bf16", ids="i64", scale=64.0, padding=0.01),
        # a short uneven batch into a small 32-bit table
        dict(name="embedding_grad_short", kind="embedding_grad", ranks=4, tokens=517, ragged=True, vocab=8009,
             width=1000, type="f32", out="f32", ids="i64", scale=1.0, padding=0.05, accumulate=False),
        # a training step's tokens, common ones thousands of times, into 32-bit gradients of the whole table
        dict(name="embedding_grad_train", kind="embedding_grad", ranks=8, tokens=8192, ragged=False, vocab=32000,
             width=4096, type="bf16", out="f32", ids="i64", scale=64.0, padding=0.01, accumulate=False),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "dispatch", "combine", "embedding", "embedding_grad"])
    ranks = rng.choice([1, 2, 3, 4, 8, 16])
    case = dict(kind=kind, ranks=ranks, ragged=rng.random() < 0.5, type=rng.choice(["f32", "bf16", "f16"]),
                padding=rng.choice([0.0, 0.0, 0.01, 0.2]))
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _spread(rng, 8, 512 // groups)
        case.update(grad=rng.random() < 0.5, tokens=max(1, _spread(rng, 1, 65536) // ranks), experts=experts,
                    top_groups=rng.randint(1, groups), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, group_by=rng.choice(["max", "top2"]),
                    renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
        case["top_k"] = rng.randint(1, min(12, case["top_groups"] * (experts // groups)))
        return case
    width = _spread(rng, 64, 8192)
    if rng.random() < 0.7:
        width = max(64, width // 64 * 64)
    case["width"] = width
    if kind in ("dispatch", "combine"):
        top_k = rng.randint(1, 10)
        # at most 2**27 values moved to the experts
        most = max(1, min(32768, 2**27 // (width * top_k)))
        case.update(tokens=max(1, _spread(rng, 1, most) // ranks), experts=ranks * _spread(rng, 1, 256 // ranks),
                    top_k=top_k, room=rng.choice([1.0, 1.5, 4.0]))
        case["top_k"] = min(top_k, case["experts"])
        if kind == "combine":
            case["grad"] = rng.random() < 0.5
        return case
    vocab = _spread(rng, 1000, 64000)
    # tables of at most 2**27 values, looked up at most 2**27 / width times
    case.update(vocab=min(vocab, 2**27 // width), tokens=max(1, _spread(rng, 1, min(65536, 2**27 // width)) // ranks),
                ids=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 0.5, math.sqrt(width)]))
    if kind == "embedding_grad":
        case.update(out=rng.choice(["f32", case["type"]]), accumulate=rng.random() < 0.4)
    return case


def _tokens(case):
    """Tokens of each rank; ragged: fewer on later ranks, down to almost none."""
    R, t = case["ranks"], case["tokens"]
    if not case["ragged"]:
        return [t] * R
    return [t - (t * r * r) // (R * R) for r in range(R)]


def _room(case):
    """Rows that each expert rank has room for."""
    entries = sum(_tokens(case)) * case["top_k"]
    return max(1, int(math.ceil(case["room"] * entries / case["ranks"])))


def _split(case, vocab):
    """The vocabulary rows of each rank: segments of ceil(V / R)."""
    R = case["ranks"]
    s = -(-vocab // R)
    return [max(0, min((c + 1) * s, vocab) - c * s) for c in range(R)]


_ranks_open = None


def _session(ranks):
    """The process's session, opened for `ranks` ranks."""
    global _ranks_open
    if _ranks_open == ranks:
        return
    import rank_reductions_amd as rr
    rr.reset()
    rr.register(ranks, device=torch.cuda.current_device())
    _ranks_open = ranks


def _choices(case, g, dev):
    """Distinct experts for every token, some experts more popular than others, padding tokens with none."""
    E, K = case["experts"], case["top_k"]
    pop = torch.randn(E, generator=g, device=dev) * 0.5
    out = []
    for t in _tokens(case):
        e = torch.argsort(torch.randn(t, E, generator=g, device=dev) + pop, dim=1, descending=True)[:, :K]
        gone = torch.rand(t, generator=g, device=dev) < case["padding"]
        out.append(torch.where(gone[:, None], -1, e).to(torch.int32).contiguous())
    return out


def _buffers(R, C, D, dt, dev):
    """The ranks' row buffers, C rows each, one after the other, and a row behind them for what has no place."""
    buffer = torch.zeros(R * C + 1, D, dtype=dt, device=dev)
    return buffer, list(buffer[:R * C].view(R, C, D))


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = TYPES[case["type"]]
    R, T, kind = case["ranks"], _tokens(case), case["kind"]
    st = {"case": case}

    def normal(*shape, of=dt, std=1.0):
        x = torch.empty(*shape, dtype=of, device=dev)
        x.normal_(0.0, std, generator=g)
        return x

    if kind == "route":
        E, K = case["experts"], case["top_k"]
        st["logits"] = []
        for t in T:
            l = normal(t, E, std=1.5)
            gone = torch.rand(t, generator=g, device=dev) < case["padding"]
            st["logits"].append(l.masked_fill_(gone[:, None], -math.inf))
        st["bias"] = normal(E, of=torch.float32, std=0.05) if case["bias"] else None
        st["d_weights"] = [normal(t, K, of=torch.float32) for t in T]
        st["weights"] = [torch.empty(t, K, dtype=torch.float32, device=dev) for t in T]
        st["chosen"] = [torch.empty(t, K, dtype=torch.int32, device=dev) for t in T]
        st["d_logits"] = [torch.empty_like(l) for l in st["logits"]]
    elif kind in ("dispatch", "combine"):
        D, C = case["width"], _room(case)
        st["experts"] = _choices(case, g, dev)
        if kind == "dispatch":
            st["xs"] = [normal(t, D) for t in T]
            st["buffer"], st["rows"] = _buffers(R, C, D, dt, dev)
        else:
            st["buffer"], st["rows"] = _buffers(R, C, D, dt, dev)
            for x in st["rows"]:
                x.normal_(0.0, 1.0, generator=g)
            st["weights"] = [torch.rand(t, case["top_k"], generator=g, device=dev) for t in T]
            st["outs"] = [torch.empty(t, D, dtype=dt, device=dev) for t in T]
            if case["grad"]:
                st["d_outs"] = [normal(t, D) for t in T]
                st["d_buffer"], st["d_rows"] = _buffers(R, C, D, dt, dev)
                st["d_weights"] = [torch.empty(t, case["top_k"], dtype=torch.float32, device=dev) for t in T]
    else:
        V, D = case["vocab"], case["width"]
        st["ids"] = []
        for t in T:
            # token counts fall off as one over the id, as in a vocabulary sorted by frequency
            u = torch.rand(t, generator=g, device=dev, dtype=torch.float64)
            i = (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1)
            gone = torch.rand(t, generator=g, device=dev) < case["padding"]
            st["ids"].append(torch.where(gone, -1, i).to(torch.int32 if case["ids"] == "i32" else torch.int64))
        if kind == "embedding":
            st["tables"] = [normal(v, D, std=0.02) for v in _split(case, V)]
            st["outs"] = [torch.empty(t, D, dtype=dt, device=dev) for t in T]
        else:
            st["d_outs"] = [normal(t, D, std=0.1) for t in T]
            st["d_tables"] = [torch.empty(v, D, dtype=TYPES[case["out"]], device=dev) for v in _split(case, V)]
            if case["accumulate"]:
                st["held"] = [normal(v, D, of=TYPES[case["out"]]) for v in _split(case, V)]
    if own:
        _session(R)
        if kind == "combine":
            import rank_reductions_amd as rr
            st["plan"] = rr.dispatch_plan(st["experts"], case["experts"], capacity=_room(case))
        elif kind == "embedding_grad" and case["accumulate"]:
            for d, h in zip(st["d_tables"], st["held"]):
                d.copy_(h)
    elif kind == "combine":
        st["slots"] = _plain_plan(case, st["experts"])[0]
    return st


def run(st):
    return (_run_own if own else _run_plain)(st["case"], st)


# ---------------------------------------------------------------- the framework's operators

def _run_own(case, st):
    import rank_reductions_amd as rr
    _session(case["ranks"])
    kind = case["kind"]
    if kind == "route":
        w, e = rr.route(st["logits"], case["top_k"], score=case["score"], bias=st["bias"], groups=case["groups"],
                        top_groups=case["top_groups"], group_by=case["group_by"], renormalize=case["renormalize"],
                        scale=case["scale"], out=(st["weights"], st["chosen"]))
        if not case["grad"]:
            return w, e
        return w, e, rr.route_grad(st["logits"], e, st["d_weights"], score=case["score"],
                                   renormalize=case["renormalize"], scale=case["scale"], out=st["d_logits"])
    if kind == "dispatch":
        plan = rr.dispatch_plan(st["experts"], case["experts"], capacity=_room(case))
        rows = rr.dispatch(st["xs"], plan, out=st["rows"])
        return rows, plan.slots, plan.offsets, plan.counts
    if kind == "combine":
        y = rr.combine(st["rows"], st["plan"], st["weights"], out=st["outs"])
        if not case["grad"]:
            return y
        return y, rr.combine_grad(st["d_outs"], st["rows"], st["plan"], st["weights"],
                                  out=(st["d_rows"], st["d_weights"]))
    if kind == "embedding":
        return rr.embedding(st["ids"], st["tables"], scale=case["scale"], out=st["outs"])
    if case["accumulate"]:
        # the gradients that the program already holds, made again for each pass
        for d, h in zip(st["d_tables"], st["held"]):
            d.copy_(h)
    return rr.embedding_grad(st["ids"], st["d_outs"], case["vocab"], scale=case["scale"], out=st["d_tables"],
                             accumulate=case["accumulate"])


# ---------------------------------------------------------------- plain forms

def _plain_route(case, l, bias):
    """Scores and choices in 64 bits: which expert is chosen hangs on values next to a border."""
    T, E, K, G = l.shape[0], case["experts"], case["top_k"], case["groups"]
    x = l.double()
    if case["score"] == "softmax":
        m = x.amax(1, keepdim=True)
        s = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    c = s if bias is None else s + bias.double()
    c = torch.where(torch.isneginf(x) | torch.isnan(c), -math.inf, c)
    if G > 1:
        by_group = c.view(T, G, E // G)
        top = torch.sort(by_group, dim=2, descending=True)[0]
        score = top[:, :, 0]
        if case["group_by"] == "top2" and E // G > 1:
            score = score + top[:, :, 1]
        order = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        c = torch.where(keep[:, :, None], by_group, -math.inf).view(T, E)
    best, e = torch.sort(c, dim=1, descending=True, stable=True)
    best, e = best[:, :K], e[:, :K]
    none = torch.isneginf(best)
    w = torch.where(none, 0.0, torch.gather(torch.nan_to_num(s), 1, e))
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return (case["scale"] * w).float(), torch.where(none, -1, e).int()


def _plain_route_grad(case, l, e, dw):
    x = l.float()
    none = e < 0
    at = e.clamp(min=0).long()
    dw = torch.where(none, 0.0, dw * case["scale"])
    if case["score"] == "softmax":
        m = x.amax(1, keepdim=True)
        s = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        s = torch.nan_to_num(s / s.sum(1, keepdim=True))
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    chosen = torch.where(none, 0.0, torch.gather(s, 1, at))
    if case["renormalize"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, math.inf)
        dw = (dw - (dw * (chosen / total)).sum(1, keepdim=True)) / total
        dw = torch.where(none, 0.0, dw)
    ds = torch.zeros_like(x).scatter_add_(1, at, dw)
    if case["score"] == "softmax":
        dl = s * (ds - (ds * s).sum(1, keepdim=True))
    else:
        dl = ds * s * (1.0 - s)
    return dl.to(l.dtype)


def _plain_plan(case, experts):
    R, E, K, C = case["ranks"], case["experts"], case["top_k"], _room(case)
    per = E // R
    flat = torch.cat([e.reshape(-1) for e in experts]).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True)[1]
    counts = torch.bincount(key, minlength=E + 1)[:E].view(R, per)
    offsets = torch.zeros(R, per + 1, dtype=torch.long, device=flat.device)
    offsets[:, 1:] = counts.cumsum(1)
    # rows before each rank's first in the order of all experts
    before = torch.cat([counts.sum(1), counts.new_zeros(1)]).cumsum(0)
    before = torch.cat([before.new_zeros(1), before])[:R + 1]
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    place = place - before[torch.where(flat < 0, 0, flat) // per]
    place = torch.where((flat < 0) | (place >= C), -1, place).int()
    slots = [s.view(-1, K) for s in place.split([e.numel() for e in experts])]
    return slots, list(offsets.clamp(max=C).int()), list(counts.int())


def _places(case, experts, slots):
    """Where each (token, choice) lies in the buffer of all ranks' rows; the row behind them where it has no place."""
    C, per = _room(case), case["experts"] // case["ranks"]
    return torch.where(slots >= 0, experts.long() // per * C + slots.long(), case["ranks"] * C)


def _run_plain(case, st):
    """The tokens of all ranks as one batch, split at the end."""
    kind, T = case["kind"], _tokens(case)
    if kind == "route":
        l = torch.cat(st["logits"])
        w, e = _plain_route(case, l, st["bias"])
        out = list(w.split(T)), list(e.split(T))
        if not case["grad"]:
            return out
        return out + (list(_plain_route_grad(case, l, e, torch.cat(st["d_weights"])).split(T)),)
    if kind == "dispatch":
        slots, offsets, counts = _plain_plan(case, st["experts"])
        x = torch.cat(st["xs"])
        at = _places(case, torch.cat(st["experts"]), torch.cat(slots))
        for k in range(case["top_k"]):
            st["buffer"][at[:, k]] = x
        return st["rows"], slots, offsets, counts
    if kind == "combine":
        s, w, buffer = torch.cat(st["slots"]), torch.cat(st["weights"]), st["buffer"]
        at = _places(case, torch.cat(st["experts"]), s)
        held = torch.where(s >= 0, w, 0.0)
        y = torch.zeros(at.shape[0], case["width"], dtype=torch.float32, device=at.device)
        for k in range(case["top_k"]):
            y += held[:, k:k + 1] * buffer[at[:, k]].float()
        outs = list(y.to(buffer.dtype).split(T))
        if not case["grad"]:
            return outs
        dy, dw = torch.cat(st["d_outs"]).float(), torch.empty_like(w)
        for k in range(case["top_k"]):
            dw[:, k] = torch.where(s[:, k] >= 0, (dy * buffer[at[:, k]].float()).sum(1), 0.0)
            st["d_buffer"][at[:, k]] = (w[:, k:k + 1] * dy).to(buffer.dtype)
        return outs, (st["d_rows"], list(dw.split(T)))
    V, D = case["vocab"], case["width"]
    i = torch.cat(st["ids"])
    ok = (i >= 0) & (i < V)
    if kind == "embedding":
        y = torch.cat(st["tables"])[torch.where(ok, i, 0).long()].float() * case["scale"]
        return list(torch.where(ok[:, None], y, 0.0).to(TYPES[case["type"]]).split(T))
    # one row behind the table takes what lies outside it
    total = torch.zeros(V + 1, D, dtype=torch.float32, device=i.device)
    if case["accumulate"]:
        total[:V].copy_(torch.cat(st["held"]))
    total.index_add_(0, torch.where(ok, i, V).long(), torch.cat(st["d_outs"]).float() * case["scale"])
    return [x.to(TYPES[case["out"]]) for x in total[:V].split(_split(case, V))]


# ---------------------------------------------------------------- what the operators cannot do without

def work(case):
    n, b, kind = sum(_tokens(case)), SIZE[case["type"]], case["kind"]
    if kind == "route":
        E, K = case["experts"], case["top_k"]
        by = n * (E * b + K * 8) + (E * 4 if case["bias"] else 0)
        fl = n * E * 4
        if case["grad"]:
            by += n * (E * b + K * 4)
            fl += n * K * 8
        return {"bytes": by, "flops": fl}
    if kind in ("dispatch", "combine"):
        K, D = case["top_k"], case["width"]
        rows = min(n * K, case["ranks"] * _room(case))
        if kind == "dispatch":
            return {"bytes": (n + rows) * D * b + n * K * 8, "flops": 0}
        by, fl = (rows + n) * D * b + n * K * 12, 2 * rows * D
        if case["grad"]:
            by += (n + rows) * D * b + n * K * 4
            fl += 3 * rows * D
        return {"bytes": by, "flops": fl}
    V, D, i = case["vocab"], case["width"], 4 if case["ids"] == "i32" else 8
    if kind == "embedding":
        # no row of the table has to be read twice
        return {"bytes": (min(n, V) + n) * D * b + n * i, "flops": n * D}
    o = SIZE[case["out"]]
    # accumulating: the touched rows at least are read and written
    held = min(n, V) * D * o * 2 if case["accumulate"] else V * D * o
    return {"bytes": n * (D * b + i) + held, "flops": 2 * n * D}


# ---------------------------------------------------------------- exact values, from the definitions in 64 bits

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    kind, R = case["kind"], case["ranks"]
    if kind == "route":
        ws, es, grads = [], [], []
        for l, dw in zip(st["logits"], st["d_weights"]):
            w, e = _exact_route(case, l.double(), None if st["bias"] is None else st["bias"].double())
            ws.append(w)
            es.append(e.int())
            if case["grad"]:
                grads.append(_exact_route_grad(case, l.double(), e, dw.double()))
        return (ws, es, grads) if case["grad"] else (ws, es)
    if kind in ("dispatch", "combine"):
        C, per, K, D = _room(case), case["experts"] // R, case["top_k"], case["width"]
        ex = [e.cpu().numpy().astype(np.int64) for e in st["experts"]]
        counts = np.zeros(case["experts"], np.int64)
        for e in ex:
            counts += np.bincount(e[e >= 0], minlength=case["experts"])
        offsets = np.zeros((R, per + 1), np.int64)
        offsets[:, 1:] = np.cumsum(counts.reshape(R, per), 1)
        start = offsets[:, :per].reshape(-1).copy()
        slots = []
        for e in ex:
            s = np.full(e.shape, -1, np.int64)
            for x in range(case["experts"]):  # entries of one expert follow one another in token order
                at = np.nonzero(e.reshape(-1) == x)[0]
                s.reshape(-1)[at] = start[x] + np.arange(at.size)
                start[x] += at.size
            s[s >= C] = -1
            slots.append(s)
        if kind == "dispatch":
            rows = [torch.zeros(C, D, dtype=torch.float64, device=st["xs"][0].device) for _ in range(R)]
            for x, e, s in zip(st["xs"], ex, slots):
                for d in range(R):
                    t, k = np.nonzero((s >= 0) & (e // per == d))
                    rows[d][torch.from_numpy(s[t, k]).to(x.device)] = x.double()[torch.from_numpy(t).to(x.device)]
            return (rows, [torch.from_numpy(s).int() for s in slots],
                    [torch.from_numpy(o).int() for o in np.minimum(offsets, C)],
                    [torch.from_numpy(c).int() for c in counts.reshape(R, per)])
        dev = st["rows"][0].device
        outs, d_weights = [], []
        d_rows = [torch.zeros(C, D, dtype=torch.float64, device=dev) for _ in range(R)]
        for r, (e, s) in enumerate(zip(ex, slots)):
            w = st["weights"][r].double()
            y = torch.zeros(e.shape[0], D, dtype=torch.float64, device=dev)
            dw = torch.zeros(e.shape, dtype=torch.float64, device=dev)
            for d in range(R):
                t, k = np.nonzero((s >= 0) & (e // per == d))
                if not t.size:
                    continue
                at = torch.from_numpy(s[t, k]).to(dev)
                t, k = torch.from_numpy(t).to(dev), torch.from_numpy(k).to(dev)
                for lo in range(0, t.numel(), 16384):
                    a, b, c = at[lo:lo + 16384], t[lo:lo + 16384], k[lo:lo + 16384]
                    row = st["rows"][d][a].double()
                    y.index_add_(0, b, row * w[b, c][:, None])
                    if case["grad"]:
                        dy = st["d_outs"][r][b].double()
                        dw[b, c] = (dy * row).sum(1)
                        d_rows[d][a] = dy * w[b, c][:, None]
            outs.append(y)
            d_weights.append(dw)
        return (outs, (d_rows, d_weights)) if case["grad"] else outs
    V, D = case["vocab"], case["width"]
    if kind == "embedding":
        s = -(-V // R)
        outs = []
        for i in st["ids"]:
            y = torch.zeros(i.numel(), D, dtype=torch.float64, device=i.device)
            for c, table in enumerate(st["tables"]):
                at = torch.nonzero((i >= c * s) & (i < min(V, (c + 1) * s))).squeeze(1)
                y[at] = table[i[at].long() - c * s].double() * case["scale"]
            outs.append(y)
        return outs
    ids, s = torch.cat(st["ids"]).long(), -(-V // R)
    tables = []
    for c, v in enumerate(_split(case, V)):
        total = torch.zeros(v, D, dtype=torch.float64, device=ids.device)
        for i, d in zip(st["ids"], st["d_outs"]):
            at = torch.nonzero((i >= c * s) & (i < c * s + v)).squeeze(1)
            total.index_add_(0, i[at].long() - c * s, d[at].double())
        total *= case["scale"]
        tables.append(total + st["held"][c].double() if case["accumulate"] else total)
    return tables


def _exact_route(case, x, bias):
    """Choices one at a time, the best that is left each time."""
    T, E = x.shape
    G = case["groups"]
    if case["score"] == "softmax":
        s = torch.softmax(x, 1)
    else:
        s = torch.sigmoid(x)
    c = s.clone() if bias is None else s + bias
    c[torch.isneginf(x) | torch.isnan(c)] = -math.inf
    lines = torch.arange(T, device=x.device)
    if G > 1:
        v = c.reshape(T, G, -1).clone()
        first = v.max(2)
        score = first.values
        if case["group_by"] == "top2" and E // G > 1:
            v.scatter_(2, first.indices[:, :, None], -math.inf)
            score = score + v.amax(2)
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        taken = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        for _ in range(case["top_groups"]):
            left = score.masked_fill(taken, -math.inf)
            best = left.amax(1, keepdim=True)
            a = ((left == best) & ~taken).int().argmax(1)
            taken[lines, a] = True
            kept[lines, a] = True
        c = c.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    ws, es = [], []
    for _ in range(case["top_k"]):
        best = c.amax(1)
        a = (c == best[:, None]).int().argmax(1)
        none = torch.isneginf(best)
        es.append(torch.where(none, -1, a))
        ws.append(torch.where(none, 0.0, s[lines, a]))
        c[lines, a] = -math.inf
    w, e = torch.stack(ws, 1), torch.stack(es, 1)
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
    return w * case["scale"], e


def _exact_route_grad(case, x, e, dw):
    """The derivative of each weight by each logit, written out over the chosen experts."""
    none = e < 0
    at = e.clamp(min=0).long()
    if case["score"] == "softmax":
        full = torch.nan_to_num(torch.softmax(x, 1))
        p = torch.where(none, 0.0, torch.gather(full, 1, at))
    else:
        p = torch.where(none, 0.0, torch.sigmoid(torch.gather(x, 1, at)))
    g = torch.where(none, 0.0, dw) * case["scale"]
    out = torch.zeros_like(x)
    if case["renormalize"]:
        total = p.sum(1, keepdim=True)
        q = torch.where(total > 0, p / total.clamp(min=1e-300), 0.0)
        d = q * (g - (g * q).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            d = d * torch.where(none, 0.0, torch.sigmoid(-torch.gather(x, 1, at)))
        return out.scatter_add_(1, at, d)
    if case["score"] == "sigmoid":
        d = g * p * torch.where(none, 0.0, torch.sigmoid(-torch.gather(x, 1, at)))
        return out.scatter_add_(1, at, d)
    out.scatter_add_(1, at, g * p)
    return out - full * (g * p).sum(1, keepdim=True)
