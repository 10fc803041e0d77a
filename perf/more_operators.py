"""The block operators' timed cases, each with its plain form in elementary
torch operations: root-mean-square norm with the residual's addition, its
output in 8 bits and its gradient; a whole mixture-of-experts layer for a few
tokens; gradient norms and the AdamW step over many tensors at once.

`own` selects the framework's kernels instead of the plain forms.  R logical
ranks hold their tokens, or their parameters, in R tensors or maps; experts are
split over the same ranks in order.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MOST = 448.0
LEAST = 2.0 ** -117  # a row, group or block whose largest value is below this is held as zeros
GROUP = 128          # elements that share a scale of the norm's 8-bit output
BLOCK = 256          # elements that share a scale of the optimizer's 8-bit states
EPS = 1e-6
BETAS, ADAM_EPS = (0.9, 0.999), 1e-8


def listed():
    return [
        # one decoding step of 64 sequences spread over 8 ranks: the layer's output joins the residual stream
        dict(name="norm_decode", kind="norm", ranks=8, tokens=8, ragged=False, width=4096, type="bf16", weights="bf16",
             residual=True, bits=16, group=0, grad=False),
        # an uneven prompt batch, rows of an odd width in 8 bits with a scale for each group, float32 weights
        dict(name="norm_prompt_8bit", kind="norm", ranks=4, tokens=2049, ragged=True, width=5003, type="f16",
             weights="f32", residual=True, bits=8, group=GROUP, grad=False),
        # a training step's tokens of the transformer's hidden size, forward and backward
        dict(name="norm_train", kind="norm", ranks=8, tokens=2048, ragged=False, width=4096, type="bf16",
             weights="bf16", residual=True, bits=16, group=0, grad=True),
        # one sequence's next token, weights of 16 bits
        dict(name="moe_token", kind="moe", ranks=1, tokens=1, ragged=False, experts=64, top_k=8, width=4096, inner=1536,
             type="bf16", weights="bf16", out="bf16", padding=0.0),
        # an uneven handful of tokens, 32-bit rows and weights of odd sizes
        dict(name="moe_odd", kind="moe", ranks=4, tokens=3, ragged=True, experts=12, top_k=2, width=1001, inner=517,
             type="f32", weights="f32", out="f32", padding=0.0),
        # one decoding step of 64 sequences spread over 8 ranks: rows from the norm and weights in 8 bits
        dict(name="moe_decode_8bit", kind="moe", ranks=8, tokens=8, ragged=False, experts=64, top_k=8, width=4096,
             inner=1536, type="e4m3", weights="e4m3", out="bf16", padding=0.0),
        # a decoding step of 256 sequences, some of them ended
        dict(name="moe_decode_wide", kind="moe", ranks=8, tokens=32, ragged=False, experts=64, top_k=8, width=4096,
             inner=1536, type="bf16", weights="bf16", out="bf16", padding=0.1),
        # the two ranks' copies of a small float32 model, clipped by the norm of their gradients
        dict(name="adamw_small", kind="adamw", ranks=2, layers=2, width=100, inner=257, params="f32", grads="f32",
             bits=32, clip=True),
        # many small tensors: 16-bit parameters with 32-bit copies, states of 8 bits, odd sizes
        dict(name="adamw_many_8bit", kind="adamw", ranks=4, layers=24, width=251, inner=1003, params="bf16",
             grads="f32", bits=8, clip=True),
        # a few layers of the transformer, float32, one copy for each of two ranks
        dict(name="adamw_train", kind="adamw", ranks=2, layers=1, width=4096, inner=11008, params="f32", grads="f32",
             bits=32, clip=False),
        # the same layers in bfloat16 with states of 8 bits, clipped
        dict(name="adamw_train_8bit", kind="adamw", ranks=2, layers=1, width=4096, inner=11008, params="bf16",
             grads="bf16", bits=8, clip=True),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "moe", "adamw"])
    ranks = rng.choice([1, 2, 3, 4, 8])
    case = dict(kind=kind, ranks=ranks)
    if kind == "norm":
        width = _spread(rng, 64, 16384)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        t = rng.choice(["f32", "bf16", "f16"])
        # at most 2**27 bytes of rows
        tokens = max(1, _spread(rng, 1, min(65536, 2**27 // (SIZE[t] * width))) // ranks)
        grad = rng.random() < 0.4
        bits = 16 if grad or rng.random() < 0.5 else 8
        case.update(tokens=tokens, ragged=rng.random() < 0.5, width=width, type=t, weights=rng.choice([t, "f32"]),
                    residual=rng.random() < 0.7, bits=bits, group=rng.choice([0, GROUP]) if bits == 8 else 0, grad=grad)
    elif kind == "moe":
        width, inner = _spread(rng, 128, 8192), _spread(rng, 64, 4096)
        if rng.random() < 0.7:
            width, inner = max(128, width // 64 * 64), max(64, inner // 64 * 64)
        t = rng.choice(["bf16", "bf16", "f16", "f32", "e4m3", "e4m3"])
        w = "e4m3" if t == "e4m3" or (t != "f32" and rng.random() < 0.4) else t
        # at most 2**31 bytes of weights
        most = max(ranks, min(256, 2**31 // (SIZE[w] * width * inner * 3)))
        experts = _spread(rng, ranks, most) // ranks * ranks
        top_k = min(rng.randint(1, 10), experts)
        case.update(tokens=max(1, _spread(rng, 1, 2048 // top_k) // ranks), ragged=rng.random() < 0.5, experts=experts,
                    top_k=top_k, width=width, inner=inner, type=t, weights=w,
                    out=rng.choice(["bf16", "f16"]) if t == "e4m3" else t, padding=rng.choice([0.0, 0.0, 0.2]))
    else:
        width, inner = _spread(rng, 32, 4096), _spread(rng, 32, 11008)
        per = 4 * width * width + 3 * width * inner
        p = rng.choice(["f32", "bf16", "f16"])
        # at most 2**28 values on all ranks, 40 layers of nine tensors on each
        ranks = min(ranks, 2**28 // per)
        layers = min(40, _spread(rng, 1, 2**28 // (per * ranks)))
        case.update(ranks=ranks, layers=layers, width=width, inner=inner, params=p, grads=rng.choice([p, "f32"]),
                    bits=rng.choice([8, 32]), clip=rng.random() < 0.6)
    return case


def _tokens(case):
    """Tokens of each rank; ragged: fewer on later ranks, down to almost none."""
    R, t = case["ranks"], case["tokens"]
    if not case["ragged"]:
        return [t] * R
    return [t - (t * r * r) // (R * R) for r in range(R)]


def _shapes(case):
    """The parameters of a rank: nine tensors a layer."""
    w, i = case["width"], case["inner"]
    return ([(w,)] + [(w, w)] * 4 + [(w,)] + [(i, w)] * 2 + [(w, i)]) * case["layers"]


def _starts(case):
    """Where each parameter lies in a rank's flat buffer, each on a multiple of BLOCK elements, and the buffer's size."""
    at, starts = 0, []
    for s in _shapes(case):
        starts.append(at)
        at += -(-math.prod(s) // BLOCK) * BLOCK
    return starts, at


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


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    st = {"case": case}

    def normal(*shape, of="f32", std=1.0, mean=0.0):
        x = torch.empty(*shape, dtype=torch.float32 if of in ("f32", "e4m3") else TYPES[of], device=dev)
        x.normal_(mean, std, generator=g)
        return x.clamp_(-E4M3_MOST, E4M3_MOST).to(TYPES[of]) if of == "e4m3" else x

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    if case["kind"] == "norm":
        _prepare_norm(case, st, normal, uniform, dev)
    elif case["kind"] == "moe":
        _prepare_moe(case, st, normal, uniform, dev)
    else:
        _prepare_adamw(case, st, normal, uniform, dev)
    return st


def _prepare_norm(case, st, normal, uniform, dev):
    T, D, t = _tokens(case), case["width"], case["type"]
    # a residual stream with a few channels far larger than the rest, as models grow them
    outlier = 1.0 + 20.0 * (uniform(D) < 0.002)
    st["xs"] = [(normal(n, D) * outlier).to(TYPES[t]) for n in T]
    st["residuals"] = [(3.0 * normal(n, D) * outlier).to(TYPES[t]) for n in T] if case["residual"] else None
    w = normal(D, std=0.2, mean=1.0).to(TYPES[case["weights"]])
    st["weights"] = [w.clone() for _ in T]
    st["ys"] = [torch.empty(n, D, dtype=TYPES["e4m3" if case["bits"] == 8 else t], device=dev) for n in T]
    groups = -(-D // case["group"]) if case["group"] else 1
    st["scales"] = [torch.empty(n, groups, device=dev) for n in T] if case["bits"] == 8 else None
    st["sums"] = [torch.empty(n, D, dtype=TYPES[t], device=dev) for n in T] if case["residual"] else None
    if case["grad"]:
        st["d_ys"] = [normal(n, D, of=t) for n in T]
        st["d_sums"] = [normal(n, D, of=t) for n in T] if case["residual"] else None
        st["d_xs"] = [torch.empty(n, D, dtype=TYPES[t], device=dev) for n in T]
        st["d_weights"] = [torch.empty(D, dtype=TYPES[case["weights"]], device=dev) for _ in T]


def _prepare_moe(case, st, normal, uniform, dev):
    R, T, E, K, H, I = case["ranks"], _tokens(case), case["experts"], case["top_k"], case["width"], case["inner"]
    t, w = case["type"], case["weights"]
    st["xs"] = [normal(n, H, of=t, std=100.0 if t == "e4m3" else 1.0) for n in T]
    st["scales"] = [0.005 + 0.01 * uniform(n, 1) for n in T] if t == "e4m3" else None
    # 8-bit weights: codes of a normal distribution, a scale for each row
    eight = w == "e4m3"
    st["gate_up"] = [normal(E // R, 2 * I, H, of=w, std=100.0 if eight else H**-0.5) for _ in range(R)]
    st["down"] = [normal(E // R, H, I, of=w, std=100.0 if eight else I**-0.5) for _ in range(R)]
    st["gate_up_scales"] = [(0.5 + uniform(E // R, 2 * I)) * (0.01 * H**-0.5) for _ in range(R)] if eight else None
    st["down_scales"] = [(0.5 + uniform(E // R, H)) * (0.01 * I**-0.5) for _ in range(R)] if eight else None
    # some experts more popular than others; padding tokens have none
    popular = 0.5 * normal(E)
    st["experts"], st["weights"] = [], []
    for n in T:
        l = normal(n, E) + popular
        e = torch.argsort(l, dim=1, descending=True)[:, :K]
        p = torch.softmax(torch.gather(l, 1, e), 1)
        gone = (uniform(n) < case["padding"])[:, None]
        st["experts"].append(torch.where(gone, -1, e).to(torch.int32).contiguous())
        st["weights"].append(torch.where(gone, 0.0, p).contiguous())
    st["ys"] = [torch.empty(n, H, dtype=TYPES[case["out"]], device=dev) for n in T]


def _prepare_adamw(case, st, normal, uniform, dev):
    R, (starts, N), shapes = case["ranks"], _starts(case), _shapes(case)
    sizes = [math.prod(s) for s in shapes]
    # flat buffers of all ranks' values; what lies between two parameters is zero
    real = torch.zeros(N, dtype=torch.bool, device=dev)
    for a, n in zip(starts, sizes):
        real[a:a + n] = True

    def flat(std, dt="f32"):
        return (normal(R, N, std=std) * real).to(TYPES[dt])

    value = flat(0.02)
    # gradients, and states to match them: sizes differ from one stretch of 64 values to the next
    size = 1e-3 * torch.exp(1.5 * normal(R, N // 64)).repeat_interleave(64, 1)
    st["grads"] = (flat(1.0) * size).to(TYPES[case["grads"]])
    m = flat(0.3) * size
    v = (size * (0.5 + uniform(R, N))) ** 2 * real
    del size
    st["params"] = value.to(TYPES[case["params"]])
    st["master"] = value if case["params"] != "f32" else None
    st["step"] = torch.full((R,), 100, dtype=torch.int32, device=dev) + torch.arange(R, device=dev, dtype=torch.int32)
    if case["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        blocks = m.view(R, -1, BLOCK), torch.sqrt(v).view(R, -1, BLOCK)
        for name, b in zip(("m", "v"), blocks):
            s = b.abs().amax(2, keepdim=True) / E4M3_MOST
            st[name] = (b / torch.where(s > 0, s, 1.0)).clamp(-E4M3_MOST, E4M3_MOST).to(TYPES["e4m3"]).view(R, N)
            st[name + "_scale"] = s.view(R, -1)
    # what the step writes: the parameters and the state after it
    st["new"] = {k: torch.zeros_like(st[k]) for k in ("params", "master", "m", "v", "m_scale", "v_scale", "step")
                 if st.get(k) is not None}
    st["norms"] = torch.zeros(R, device=dev) if case["clip"] else None
    st["max_norm"] = 0.5 * float(1e-3 * math.exp(2.25) * math.sqrt(sum(sizes)))
    # each value's place in its parameter
    st["place"] = torch.arange(N, device=dev)
    for a, n in zip(starts, sizes):
        st["place"][a:a + -(-n // BLOCK) * BLOCK] -= a
    if own:
        import rank_reductions_amd as rr

        def maps(x, blocks=False):
            if blocks:
                return [{i: row[a // BLOCK:a // BLOCK - (-n // BLOCK)] for i, (a, n) in enumerate(zip(starts, sizes))}
                        for row in x]
            return [{i: row[a:a + n].view(s) for i, (a, n, s) in enumerate(zip(starts, sizes, shapes))} for row in x]

        def state(of):
            scales = {k: maps(of[k], True) for k in ("m_scale", "v_scale") if k in of}
            return rr.AdamWState(maps(of["params"]), case["bits"], maps(of["m"]), maps(of["v"]), of["step"],
                                 master=maps(of["master"]) if of.get("master") is not None else None, **scales)

        _session(R)
        st["maps"] = dict(grads=maps(st["grads"]), state=state(st), new=state(st["new"]))


def run(st):
    return (_run_own if own else _run_plain)(st["case"], st)


# ---------------------------------------------------------------- the framework's operators

def _run_own(case, st):
    import rank_reductions_amd as rr
    _session(case["ranks"])
    if case["kind"] == "norm":
        out = tuple(x for x in (st["ys"], st["scales"], st["sums"]) if x is not None)
        y = rr.rms_norm(st["xs"], st["weights"], eps=EPS, residuals=st["residuals"],
                        quantize="e4m3" if case["bits"] == 8 else None, group=case["group"] or None,
                        out=out if len(out) > 1 else out[0])
        if not case["grad"]:
            return y
        return y, rr.rms_norm_grad(st["d_ys"], st["sums"] if case["residual"] else st["xs"], st["weights"], eps=EPS,
                                   d_sums=st["d_sums"], out=(st["d_xs"], st["d_weights"]))
    if case["kind"] == "moe":
        return rr.moe_layer(st["xs"], st["weights"], st["experts"], st["gate_up"], st["down"], scales=st["scales"],
                            gate_up_scales=st["gate_up_scales"], down_scales=st["down_scales"],
                            dtype=TYPES[case["out"]], out=st["ys"])
    m = st["maps"]
    norms = rr.grad_norm(m["grads"], out=st["norms"]) if case["clip"] else None
    # into other buffers than the state's own, so that a pass can be made again
    rr.adamw_step(m["state"], m["grads"], lr=1e-3, betas=BETAS, eps=ADAM_EPS, weight_decay=0.1,
                  norms=norms, max_norm=st["max_norm"] if case["clip"] else None, seed=5, out=m["new"])
    return dict(st["new"], norms=norms) if case["clip"] else st["new"]


# ---------------------------------------------------------------- plain forms

def _run_plain(case, st):
    return {"norm": _plain_norm, "moe": _plain_moe, "adamw": _plain_adamw}[case["kind"]](case, st)


def _plain_quantize(y, group):
    """Values in 8 bits, with a scale for each group of consecutive ones in a row (0: for the row)."""
    T, D = y.shape
    group = group or D
    groups = -(-D // group)
    padded = torch.zeros(T, groups * group, dtype=y.dtype, device=y.device)
    padded[:, :D] = y
    most = padded.view(T, groups, group).abs().amax(2)
    none = most < LEAST
    factor = torch.where(none, 0.0, E4M3_MOST / torch.where(none, 1.0, most))
    codes = (padded.view(T, groups, group) * factor[:, :, None]).view(T, -1)[:, :D].to(TYPES["e4m3"])
    return codes, torch.where(none, 0.0, most / E4M3_MOST)


def _plain_norm(case, st):
    """The tokens of all ranks as one batch (they hold the same weights), split at the end."""
    T, dt = _tokens(case), TYPES[case["type"]]
    w = st["weights"][0].float()
    s = torch.cat(st["xs"])
    if case["residual"]:
        s = (s.float() + torch.cat(st["residuals"]).float()).to(dt)
    x = s.float()
    scale = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    y = x * scale * w
    out = ()
    if case["bits"] == 8:
        codes, scales = _plain_quantize(y, case["group"])
        out = (list(codes.split(T)), list(scales.split(T)))
    else:
        out = (list(y.to(dt).split(T)),)
    if case["residual"]:
        out += (list(s.split(T)),)
    out = out if len(out) > 1 else out[0]
    if not case["grad"]:
        return out
    dy = torch.cat(st["d_ys"]).float()
    n = x * scale
    dn = dy * w
    dx = scale * (dn - n * (dn * n).mean(1, keepdim=True))
    if case["residual"]:
        dx = dx + torch.cat(st["d_sums"]).float()
    dw = [p.sum(0).to(st["weights"][0].dtype) for p in (dy * n).split(T)]
    return out, (list(dx.to(dt).split(T)), dw)


def _plain_moe(case, st):
    """Each choice with its expert's weights gathered, or where choices are more than experts each expert on all tokens."""
    T, K, E, I = _tokens(case), case["top_k"], case["experts"], case["inner"]
    per = E // case["ranks"]
    x = torch.cat(st["xs"]).float()
    if st["scales"] is not None:
        x = x * torch.cat(st["scales"])
    e, p = torch.cat(st["experts"]).long(), torch.cat(st["weights"])
    eight = st["gate_up_scales"] is not None

    def weights(name, r, at):
        w = st[name][r][at].float()
        return w * st[name + "_scales"][r][at][..., None] if eight else w

    if case["ranks"] == 1 and e.numel() <= E:
        at = e.reshape(-1).clamp(min=0)
        a = weights("gate_up", 0, at) @ x.repeat_interleave(K, 0)[:, :, None]
        a = a[:, :I] / (1.0 + torch.exp(-a[:, :I])) * a[:, I:]
        y = (weights("down", 0, at) @ a).view(-1, K, case["width"])
        y = (torch.where(e < 0, 0.0, p)[:, :, None] * y).sum(1)
    else:
        y = torch.zeros(x.shape[0], case["width"], device=x.device)
        for i in range(E):
            a = x @ weights("gate_up", i // per, i % per).t()
            a = a[:, :I] / (1.0 + torch.exp(-a[:, :I])) * a[:, I:]
            y += torch.where(e == i, p, 0.0).sum(1, keepdim=True) * (a @ weights("down", i // per, i % per).t())
    return list(y.to(TYPES[case["out"]]).split(T))


def _mix(x):
    """32 bits scrambled: products with odd numbers from the digits of the golden ratio and of the roots of 2 and 3."""
    x = (x * 0x9E3779B9) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _plain_adamw(case, st):
    R = case["ranks"]
    g = st["grads"].float()
    out = {"step": st["step"] + 1}
    if case["clip"]:
        norms = torch.sqrt(st["grads"].double().square().sum(1)).float()
        out["norms"] = norms
        g = g * torch.where(norms > st["max_norm"], st["max_norm"] / norms, 1.0)[:, None]
    t = out["step"].double()[:, None]
    (b1, b2), lr = BETAS, 1e-3
    c1, c2 = (lr / (1.0 - b1 ** t)).float(), (1.0 / torch.sqrt(1.0 - b2 ** t)).float()
    m, v = st["m"], st["v"]
    if case["bits"] == 8:
        m = (m.float().view(R, -1, BLOCK) * st["m_scale"][:, :, None]).view(R, -1)
        v = (v.float().view(R, -1, BLOCK) * st["v_scale"][:, :, None]).view(R, -1).square()
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * (g * g)
    p = st["params"] if st["master"] is None else st["master"]
    p = p * (1.0 - lr * 0.1) - c1 * m / (torch.sqrt(v) * c2 + ADAM_EPS)
    out["params"] = p.to(st["params"].dtype)
    if st["master"] is not None:
        out["master"] = p
    if case["bits"] == 32:
        out["m"], out["v"] = m, v
        return out
    out["m"], out["m_scale"] = (x.view(R, -1) for x in _plain_quantize(m.view(-1, BLOCK), 0))
    # the root of v, rounded up or down by chance: small changes of a long mean would be lost otherwise
    r = torch.sqrt(v).view(R, -1, BLOCK)
    most = r.amax(2)
    none = most < LEAST
    x = r * torch.where(none, 0.0, E4M3_MOST / torch.where(none, 1.0, most))[:, :, None]
    h = _mix((_mix(_mix(out["step"].long()) + 5)[:, None] + (st["place"] >> 1)) & 0xFFFFFFFF)
    chance = torch.where(st["place"] % 2 == 1, h >> 16, h & 0xFFFF).view(R, -1, BLOCK).double() / 65536
    x = x.clamp(max=E4M3_MOST).double()
    grid = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    q = (torch.floor(x / grid + chance) * grid).clamp(max=E4M3_MOST)
    q = torch.where(x > 0, q.clamp(min=2.0 ** -9), 0.0)
    out["v"], out["v_scale"] = q.float().to(TYPES["e4m3"]).view(R, -1), torch.where(none, 0.0, most / E4M3_MOST)
    return out


# ---------------------------------------------------------------- what the operators cannot do without

def work(case):
    if case["kind"] == "norm":
        n, D, b, w = sum(_tokens(case)), case["width"], SIZE[case["type"]], SIZE[case["weights"]]
        by = n * D * (b * (3 if case["residual"] else 1) + (1 if case["bits"] == 8 else b)) + case["ranks"] * D * w
        if case["bits"] == 8:
            by += n * 4 * (-(-D // case["group"]) if case["group"] else 1)
        if case["grad"]:
            by += n * D * b * (4 if case["residual"] else 3) + 2 * case["ranks"] * D * w
        return {"bytes": by, "flops": n * D * (15 if case["grad"] else 5)}
    if case["kind"] == "moe":
        n, K, E, H, I = sum(_tokens(case)), case["top_k"], case["experts"], case["width"], case["inner"]
        b = SIZE[case["weights"]]
        # the experts that some token is expected to choose, were all alike popular
        chosen = E * (1.0 - (1.0 - K / E) ** n)
        by = chosen * (3 * H * I * b + ((2 * I + H) * 4 if b == 1 else 0))
        by += n * (H * (SIZE[case["type"]] + SIZE[case["out"]]) + K * 8 + (4 if case["type"] == "e4m3" else 0))
        return {"bytes": by, "flops": n * K * 6 * H * I}
    n = case["ranks"] * sum(math.prod(s) for s in _shapes(case))
    p, g = SIZE[case["params"]], SIZE[case["grads"]]
    by = n * (8 + (p if p < 4 else 0) + g * (2 if case["clip"] else 1))
    by += n * 16 if case["bits"] == 32 else n * 4 + n * 16 // BLOCK
    return {"bytes": by, "flops": n * (20 if case["bits"] == 8 else 14)}


# ---------------------------------------------------------------- exact values, from the definitions in 64 bits

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    return {"norm": _exact_norm, "moe": _exact_moe, "adamw": _exact_adamw}[case["kind"]](case, st)


def _exact_norm(case, st):
    """Rank by rank; the norm is that of the sums as they are stored.  8-bit values before their rounding."""
    dt, D = TYPES[case["type"]], case["width"]
    ys, scales, sums, dxs, dws = [], [], [], [], []
    for r, x in enumerate(st["xs"]):
        s = x.double()
        if case["residual"]:
            s = s + st["residuals"][r].double()
            sums.append(s)
            s = s.to(dt).double()
        w = st["weights"][r].double()
        root = torch.sqrt(s.square().sum(1) / D + EPS)[:, None]
        y = s / root * w
        if case["bits"] == 8:
            group = case["group"] or D
            parts = y.split(group, 1)
            most = torch.stack([p.abs().amax(1) for p in parts], 1) if y.shape[0] else y.new_zeros(0, len(parts))
            safe = torch.where(most > 0, most, 1.0)
            ys.append(torch.cat([p * (E4M3_MOST / safe[:, i:i + 1]) for i, p in enumerate(parts)], 1))
            scales.append(most / E4M3_MOST)
        else:
            ys.append(y)
        if case["grad"]:
            dy = st["d_ys"][r].double()
            # of sum(dy * w * s / root): by s directly, and through the root
            d = dy * w / root - s * ((dy * w * s).sum(1, keepdim=True) / (D * root ** 3))
            dxs.append(d + st["d_sums"][r].double() if case["residual"] else d)
            dws.append((dy * s / root).sum(0))
    out = tuple(x for x in (ys, scales, sums) if x)
    out = out if len(out) > 1 else out[0]
    return (out, (dxs, dws)) if case["grad"] else out


def _exact_moe(case, st):
    """Expert by expert, over the tokens that chose it."""
    T, E, I = _tokens(case), case["experts"], case["inner"]
    per = E // case["ranks"]
    if sum(T) * E * case["width"] * I > 2**40:
        return None
    x = torch.cat(st["xs"]).double()
    if st["scales"] is not None:
        x = x * torch.cat(st["scales"]).double()
    e, p = torch.cat(st["experts"]), torch.cat(st["weights"]).double()
    y = torch.zeros(x.shape[0], case["width"], dtype=torch.float64, device=x.device)
    for i in range(E):
        t, k = torch.nonzero(e == i, as_tuple=True)
        if not t.numel():
            continue
        up, down = st["gate_up"][i // per][i % per].double(), st["down"][i // per][i % per].double()
        if st["gate_up_scales"] is not None:
            up = up * st["gate_up_scales"][i // per][i % per].double()[:, None]
            down = down * st["down_scales"][i // per][i % per].double()[:, None]
        gate, lift = (x[t] @ up.t()).split(I, 1)
        y.index_add_(0, t, p[t, k][:, None] * ((gate * torch.sigmoid(gate) * lift) @ down.t()))
    return list(y.split(T))


def _exact_adamw(case, st):
    """Rank by rank; 8-bit values before their rounding."""
    out = {}

    def add(name, x):
        out.setdefault(name, []).append(x)

    for r in range(case["ranks"]):
        g, t = st["grads"][r].double(), int(st["step"][r]) + 1
        if case["clip"]:
            norm = torch.linalg.vector_norm(g)
            add("norms", norm)
            g = g * min(1.0, st["max_norm"] / float(norm))
        m, v = st["m"][r].double(), st["v"][r].double()
        if case["bits"] == 8:
            m = m * st["m_scale"][r].double().repeat_interleave(BLOCK)
            v = (v * st["v_scale"][r].double().repeat_interleave(BLOCK)) ** 2
        m.mul_(BETAS[0]).add_(g, alpha=1.0 - BETAS[0])
        v.mul_(BETAS[1]).addcmul_(g, g, value=1.0 - BETAS[1])
        p = (st["params"] if st["master"] is None else st["master"])[r].double()
        p = p - 1e-3 * (0.1 * p + m / (1.0 - BETAS[0] ** t) / (torch.sqrt(v / (1.0 - BETAS[1] ** t)) + ADAM_EPS))
        add("params", p)
        if st["master"] is not None:
            add("master", p)
        if case["bits"] == 8:
            for name, x in (("m", m), ("v", torch.sqrt(v))):
                x = x.view(-1, BLOCK)
                most = x.abs().amax(1, keepdim=True)
                add(name, (x * (E4M3_MOST / torch.where(most > 0, most, 1.0))).view(-1))
                add(name + "_scale", most.view(-1) / E4M3_MOST)
        else:
            add("m", m)
            add("v", v)
        add("step", torch.tensor(t, dtype=torch.int32))
    return {k: torch.stack(x) for k, x in out.items()}
