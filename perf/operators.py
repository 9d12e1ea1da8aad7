"""Cases of the language-model operators around the gradient all-reduce: the
global gradient norm and clipping (alone, and with the all-reduce that brings
the gradients), the embedding lookup with its gradient, and the softmax cross
entropy of a linear head over a large vocabulary with its gradients.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through ``ring_all_reduce_ar_amd``.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}
IGNORE = -100
CLIP_EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the clip of a small model's parameter gradients after an all-reduce: latency counts
        {"name": "clip small bf16", "op": "clip", "layout": "replicated", "ranks": 2, "tensors": 37, "total": 150_001,
         "packed": False, "dtype": "bf16", "norm": "l2", "max_norm": 0.1},
        # one 25 MiB data-parallel gradient bucket of ten tensors at 8 ranks: averaged and clipped in one call
        {"name": "reduce+clip bucket f32", "op": "reduce_clip", "ranks": 8, "tensors": 10, "total": 6_553_600,
         "packed": True, "dtype": "f32", "norm": "l2", "max_norm": 0.5},
        # the gradients of a large half-precision model, 256 MiB for each of 8 ranks
        {"name": "reduce+clip large f16", "op": "reduce_clip", "ranks": 8, "tensors": 29, "total": 134_217_728,
         "packed": True, "dtype": "f16", "norm": "l2", "max_norm": 4.0},
        # sharded optimizer states: each of 8 ranks holds its part of the gradient, the norm goes over all of them
        {"name": "clip shards f32", "op": "clip", "layout": "sharded", "ranks": 8, "tensors": 29, "total": 33_554_437,
         "packed": True, "dtype": "f32", "norm": "l2", "max_norm": 1.0},
        # serving: the embedding of one step's tokens of a small batch
        {"name": "lookup few bf16", "op": "lookup", "tokens": 4, "rows": 32_000, "width": 4096, "dtype": "bf16",
         "scale": 64.0, "first": 0, "index": "i64"},
        # training: the embedding of a batch, one rank's half of a vocabulary that two ranks share
        {"name": "lookup batch f16", "op": "lookup", "tokens": 16_384, "rows": 32_768, "width": 4096, "dtype": "f16",
         "scale": 1.0, "first": 32_768, "index": "i32"},
        # gradient of a middling vocabulary into fp32 master gradients, odd sizes
        {"name": "lookup grad f32 odd", "op": "lookup_grad", "tokens": 8191, "rows": 50_001, "width": 1027,
         "dtype": "bf16", "grad_dtype": "f32", "scale": 32.0, "first": 0, "index": "i64"},
        # gradient of a large vocabulary, whose all-reduce is the largest of a model's
        {"name": "lookup grad large bf16", "op": "lookup_grad", "tokens": 32_768, "rows": 131_072, "width": 4096,
         "dtype": "bf16", "grad_dtype": "bf16", "scale": 1.0, "first": 0, "index": "i64"},
        # scoring a few tokens: the whole head is read for three rows
        {"name": "loss few f16", "op": "loss", "tokens": 3, "vocab": 65_536, "width": 2048, "dtype": "f16",
         "ignored": 0.0, "index": "i64"},
        # evaluation of a batch
        {"name": "loss batch bf16", "op": "loss", "tokens": 4096, "vocab": 65_536, "width": 2048, "dtype": "bf16",
         "ignored": 0.05, "index": "i64"},
        # a training step of a small fp32 model with odd sizes: loss and both gradients
        {"name": "loss step f32 odd", "op": "loss_step", "tokens": 1021, "vocab": 32_003, "width": 770, "dtype": "f32",
         "ignored": 0.1, "index": "i32"},
        # a training step of a large model's head: loss and both gradients
        {"name": "loss step large bf16", "op": "loss_step", "tokens": 8192, "vocab": 131_072, "width": 4096,
         "dtype": "bf16", "ignored": 0.02, "index": "i64"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["clip", "reduce_clip", "lookup", "lookup_grad", "loss", "loss_step"])
    if op in ("clip", "reduce_clip"):
        ranks = rng.choice([1, 2, 3, 4, 5, 8, 16]) if op == "clip" else rng.choice([2, 3, 4, 5, 6, 7, 8, 16])
        total = min(_log_int(rng, 1000, 134_217_728), 1_073_741_824 // ranks)
        case = {"op": op, "ranks": ranks, "tensors": min(_log_int(rng, 1, 200), total), "total": total,
                "packed": rng.random() < 0.5, "dtype": rng.choice(["f32", "f16", "bf16"]),
                "norm": rng.choice(["l2", "l2", "inf"]), "max_norm": math.exp(rng.uniform(math.log(1e-3), math.log(10)))}
        if case["dtype"] == "f32":
            case["total"] = max(case["tensors"], total // 2)
        if op == "clip":
            case["layout"] = rng.choice(["replicated", "sharded"])
        return case
    if op in ("lookup", "lookup_grad"):
        case = {"op": op, "tokens": _log_int(rng, 1, 32_768), "rows": _log_int(rng, 500, 131_072),
                "width": _log_int(rng, 32, 4096), "dtype": rng.choice(["f32", "f16", "bf16"]),
                "scale": rng.choice([1.0, 0.5, 22.627417]), "first": rng.choice([0, 0, 1000]),
                "index": rng.choice(["i32", "i64"])}
        if rng.random() < 0.7:
            case["width"] = max(32, case["width"] // 32 * 32)
        if case["dtype"] == "f32":
            case["rows"] = max(500, case["rows"] // 2)
        if op == "lookup_grad":
            case["grad_dtype"] = rng.choice([case["dtype"], "f32"])
            if case["grad_dtype"] == "f32":
                case["rows"] = min(case["rows"], 65_536)
        return case
    case = {"op": op, "tokens": _log_int(rng, 1, 8192), "vocab": _log_int(rng, 500, 131_072),
            "width": _log_int(rng, 64, 4096), "dtype": rng.choice(["f16", "bf16", "bf16", "f32"]),
            "ignored": rng.choice([0.0, 0.1, 0.5]), "index": rng.choice(["i32", "i64"])}
    if rng.random() < 0.7:
        case["width"] = max(64, case["width"] // 64 * 64)
    if case["dtype"] == "f32":
        case["width"] = min(case["width"], 1024)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _sizes(case):
    """Element counts of the tensors of one rank: from small vectors to large
    matrices, log-uniform over a factor of a thousand, `total` in all."""
    n, total = case["tensors"], case["total"]
    w = [math.exp(6.9 * ((i * 0.6180339887) % 1.0)) for i in range(n)]
    c = [max(1, int(total * x / sum(w))) for x in w]
    c[c.index(max(c))] += total - sum(c)
    return c


def _views(flat, offsets, sizes):
    return [flat[o:o + s] for o, s in zip(offsets, sizes)]


def _gradients(case, g):
    """One flat buffer for each rank, its tensors at the same offsets in each:
    packed back to back, as in a bucket, or each on a 512-byte boundary, as
    separate allocations. Gradients are N(0, 1e-3^2) with 1% of outliers."""
    dt, e = DTYPE[case["dtype"]], ESIZE[case["dtype"]]
    sizes = _sizes(case)
    step = 1 if case["packed"] else 512 // e
    offsets, at = [], 0
    for s in sizes:
        offsets.append(at)
        at += -(-s // step) * step
    rows = 1 if case.get("layout") == "replicated" else case["ranks"]
    flats = []
    for _ in range(rows):
        x = torch.randn(at, generator=g, device="cuda", dtype=torch.float32).mul_(1e-3)
        x[torch.randint(0, at, (at // 100 + 1,), generator=g, device="cuda")] *= 1000.0
        flats.append(x.to(dt))
    while len(flats) < case["ranks"]:  # after an all-reduce every rank holds the same
        flats.append(flats[0].clone())
    outs = [torch.zeros(at, dtype=dt, device="cuda") for _ in range(case["ranks"])]
    send = [_views(f, offsets, sizes) for f in flats]
    recv = [_views(f, offsets, sizes) for f in outs]
    return {"send": send, "recv": recv, "outs": outs, "counts": sizes, "norm_out": torch.zeros(1, device="cuda"),
            "send_ptrs": [s[t].data_ptr() for t in range(len(sizes)) for s in send],
            "recv_ptrs": [r[t].data_ptr() for t in range(len(sizes)) for r in recv]}


def _tokens(n, rows, g):
    """Token numbers as text has them: the k-th most frequent one about 1/k as
    often as the first, spread over the rows."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    k = (torch.exp(u * math.log(rows + 1.0)) - 1.0).long().clamp_(0, rows - 1)
    return (k * 7919 + 13) % rows


INDEX = {"i32": torch.int32, "i64": torch.int64}


def _normal(g, *shape, dtype, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] in ("clip", "reduce_clip"):
        return state | _gradients(case, g)
    dt = DTYPE[case["dtype"]]
    if case["op"] in ("lookup", "lookup_grad"):
        n, rows, width = case["tokens"], case["rows"], case["width"]
        # a rank that holds rows from `first` on sees the other ranks' tokens too
        tokens = _tokens(n, rows + case["first"], g).to(INDEX[case["index"]])
        state["tokens"] = tokens
        if case["op"] == "lookup":
            state["weight"] = _normal(g, rows, width, dtype=dt, std=0.02)
            state["out"] = torch.empty(n, width, dtype=dt, device="cuda")
        else:
            state["grad_out"] = _normal(g, n, width, dtype=dt, std=1e-2)
            state["grad_weight"] = torch.empty(rows, width, dtype=DTYPE[case["grad_dtype"]], device="cuda")
        return state
    n, vocab, width = case["tokens"], case["vocab"], case["width"]
    state["hidden"] = _normal(g, n, width, dtype=dt)
    state["weight"] = _normal(g, vocab, width, dtype=dt, std=1.5 / math.sqrt(width))
    targets = _tokens(n, vocab, g)
    drop = torch.rand(n, generator=g, device="cuda") < case["ignored"]
    state["targets"] = torch.where(drop, torch.full_like(targets, IGNORE), targets).to(INDEX[case["index"]])
    state["losses"] = torch.empty(n, device="cuda")
    state["lse"] = torch.empty(n, device="cuda")
    if case["op"] == "loss_step":
        state["grad_losses"] = torch.full((n,), 1.0 / n, device="cuda")  # of the mean
        state["grad_hidden"] = torch.empty_like(state["hidden"])
        state["grad_weight"] = torch.empty_like(state["weight"])
    return state


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
_comms = {}


def _comm(state, need):
    """The program's communicator for this number of ranks, with a workspace
    that holds what this state's calls need; both are kept, as a training
    program keeps them."""
    import ring_all_reduce_ar_amd as ar
    ranks = state["case"].get("ranks", 1)
    comm, ws = _comms.get(ranks, (None, None))
    if comm is None:
        comm = ar.Comm(ranks, 0)
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        ar.ar_comm_set_workspace(comm, ws)
    _comms[ranks] = (comm, ws)
    state["ready"] = (ar, comm)
    return state["ready"]


def _run_own(state):
    case = state["case"]
    op = case["op"]
    ready = state.get("ready")
    if op in ("clip", "reduce_clip"):
        if ready is None:
            import ring_all_reduce_ar_amd as ar
            ready = _comm(state, ar.ar_clip_workspace_bytes())
        ar, comm = ready
        if op == "clip":
            ar.ar_clip_grads(comm, state["send_ptrs"], state["recv_ptrs"], state["counts"], case["max_norm"],
                             state["norm_out"], case["dtype"], case["layout"], case["norm"])
        else:
            ar.ar_all_reduce_clip(comm, state["send_ptrs"], state["recv_ptrs"], state["counts"], case["max_norm"],
                                  state["norm_out"], case["dtype"], "avg", case["norm"])
        return {"grads": state["outs"], "norm": state["norm_out"]}
    if op == "lookup":
        ar, comm = ready or _comm(state, 16)
        ar.ar_embedding(comm, state["weight"], state["tokens"], state["out"], case["tokens"], case["rows"],
                        case["width"], case["dtype"], scale=case["scale"], first_row=case["first"])
        return state["out"]
    if op == "lookup_grad":
        if ready is None:
            import ring_all_reduce_ar_amd as ar
            ready = _comm(state, ar.ar_embedding_workspace_bytes(case["tokens"], case["rows"], case["width"]))
        ar, comm = ready
        ar.ar_embedding_backward(comm, state["grad_out"], state["tokens"], state["grad_weight"], case["tokens"],
                                 case["rows"], case["width"], case["dtype"], case["grad_dtype"], scale=case["scale"],
                                 first_row=case["first"])
        return state["grad_weight"]
    step = op == "loss_step"
    if ready is None:
        import ring_all_reduce_ar_amd as ar
        ready = _comm(state, ar.ar_linear_cross_entropy_workspace_bytes(case["tokens"], case["vocab"], case["width"],
                                                                       case["dtype"], backward=step))
    ar, comm = ready
    ar.ar_linear_cross_entropy(comm, state["hidden"], state["weight"], state["targets"], state["losses"],
                               state["lse"], case["tokens"], case["vocab"], case["width"], case["dtype"],
                               ignore_index=IGNORE)
    if not step:
        return {"losses": state["losses"], "lse": state["lse"]}
    ar.ar_linear_cross_entropy_backward(comm, state["hidden"], state["weight"], state["targets"], state["lse"],
                                        state["grad_losses"], state["grad_hidden"], state["grad_weight"],
                                        case["tokens"], case["vocab"], case["width"], case["dtype"],
                                        ignore_index=IGNORE)
    return {"losses": state["losses"], "lse": state["lse"], "grad_hidden": state["grad_hidden"],
            "grad_weight": state["grad_weight"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_norm(x, kind):
    return x.double().square().sum().sqrt() if kind == "l2" else x.abs().max().double()


def _plain_clip(state):
    case = state["case"]
    dt = DTYPE[case["dtype"]]
    flats = [torch.cat([t.float() for t in s]) for s in state["send"]]
    if case["op"] == "reduce_clip":
        flats = [(torch.stack(flats).sum(0) / case["ranks"]).to(dt).float()]  # what the all-reduce gives every rank
    elif case["layout"] == "replicated":
        flats = flats[:1]
    total = _plain_norm(torch.cat(flats) if len(flats) > 1 else flats[0], case["norm"])
    scale = torch.clamp(case["max_norm"] / (total + CLIP_EPS), max=1.0).float()
    parts = [torch.split((x * scale).to(dt), state["counts"]) for x in flats] * (case["ranks"] // len(flats))
    torch._foreach_copy_([t for recv in state["recv"] for t in recv], [t for part in parts for t in part])
    return {"grads": state["outs"], "norm": total.float().reshape(1)}


def _plain_lookup(state):
    case = state["case"]
    at = state["tokens"].long() - case["first"]
    here = (at >= 0) & (at < case["rows"])
    rows = state["weight"][at.clamp(0, case["rows"] - 1)].float() * case["scale"]
    return torch.where(here[:, None], rows, torch.zeros((), device="cuda")).to(DTYPE[case["dtype"]])


def _plain_lookup_grad(state):
    case = state["case"]
    at = state["tokens"].long() - case["first"]
    here = (at >= 0) & (at < case["rows"])
    rows = torch.where(here[:, None], state["grad_out"].float(), torch.zeros((), device="cuda"))
    grad = torch.zeros(case["rows"], case["width"], device="cuda")
    grad.index_add_(0, at.clamp(0, case["rows"] - 1), rows)
    return (grad * case["scale"]).to(DTYPE[case["grad_dtype"]])


def _plain_loss(state):
    case = state["case"]
    x, w = state["hidden"].float(), state["weight"].float()
    targets = state["targets"].long()
    kept = targets != IGNORE
    at = targets.clamp(min=0)[:, None]
    logits = x @ w.t()
    top = logits.max(dim=1, keepdim=True).values
    lse = top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True))
    losses = torch.where(kept, (lse - logits.gather(1, at))[:, 0], torch.zeros((), device="cuda"))
    if case["op"] == "loss":
        return {"losses": losses, "lse": lse[:, 0]}
    d = torch.exp(logits - lse)
    del logits
    d.scatter_add_(1, at, torch.full_like(lse, -1.0))
    d *= (state["grad_losses"] * kept)[:, None]
    dt = DTYPE[case["dtype"]]
    return {"losses": losses, "lse": lse[:, 0], "grad_hidden": (d @ w).to(dt), "grad_weight": (d.t() @ x).to(dt)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("clip", "reduce_clip"):
        return _plain_clip(state)
    if op == "lookup":
        return _plain_lookup(state)
    if op == "lookup_grad":
        return _plain_lookup_grad(state)
    return _plain_loss(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _expected_rows(case):
    """About how many of the rows the tokens meet, at most."""
    return min(case["rows"], case["tokens"])


def work(case):
    op = case["op"]
    if op in ("clip", "reduce_clip"):
        size = case["total"] * ESIZE[case["dtype"]]
        inputs = 1 if op == "clip" and case["layout"] == "replicated" else case["ranks"]
        adds = inputs if op == "reduce_clip" else 0
        owned = case["ranks"] if op == "clip" and case["layout"] == "sharded" else 1
        return {"bytes": (inputs + case["ranks"]) * size, "flops": case["total"] * (adds + 3 * owned)}
    if op == "lookup":
        e, i = ESIZE[case["dtype"]], 4 if case["index"] == "i32" else 8
        moved = _expected_rows(case) * case["width"] * e + case["tokens"] * case["width"] * e
        return {"bytes": moved + case["tokens"] * i, "flops": case["tokens"] * case["width"]}
    if op == "lookup_grad":
        e, i = ESIZE[case["dtype"]], 4 if case["index"] == "i32" else 8
        return {"bytes": case["tokens"] * (case["width"] * e + i) + case["rows"] * case["width"] * ESIZE[case["grad_dtype"]],
                "flops": case["tokens"] * case["width"]}
    n, vocab, width, e = case["tokens"], case["vocab"], case["width"], ESIZE[case["dtype"]]
    step = op == "loss_step"
    operands = (n + vocab) * width * e
    return {"bytes": operands * (2 if step else 1) + n * (16 if step else 12),
            "flops": 2.0 * n * vocab * width * (3 if step else 1)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_clip(state, case):
    ranks, sizes = case["ranks"], case["counts"]
    dt = DTYPE[case["op_dtype"]]
    span = state["outs"][0].numel()
    out = [torch.zeros(span, dtype=torch.float64, device="cuda") for _ in range(ranks)]
    offsets = [(r.data_ptr() - state["outs"][0].data_ptr()) // ESIZE[case["op_dtype"]] for r in state["recv"][0]]
    square, top = 0.0, 0.0
    parts = []
    for t in range(len(sizes)):
        if case["op"] == "reduce_clip":
            acc = torch.zeros(sizes[t], dtype=torch.float64, device="cuda")
            for r in range(ranks):
                acc += state["send"][r][t]
            held = [(acc / ranks).to(torch.float32).to(dt).double()]
        elif case["layout"] == "replicated":
            held = [state["send"][0][t].double()]
        else:
            held = [state["send"][r][t].double() for r in range(ranks)]
        for h in held:
            square += float((h * h).sum())
            top = max(top, float(h.abs().max()))
        parts.append(held)
    total = math.sqrt(square) if case["norm"] == "l2" else top
    scale = min(1.0, case["max_norm"] / (total + CLIP_EPS))
    for t, held in enumerate(parts):
        for r in range(ranks):
            out[r][offsets[t]:offsets[t] + sizes[t]] = held[r if len(held) > 1 else 0] * scale
    return {"grads": out, "norm": torch.tensor([total], dtype=torch.float64)}


def _exact_lookup_grad(state, case):
    """Each row's sum by the differences of a running sum over the tokens in sorted order, a slab of columns at a time."""
    at = state["tokens"].long() - case["first"]
    keep = torch.nonzero((at >= 0) & (at < case["rows"]))[:, 0]
    order = keep[torch.argsort(at[keep], stable=True)]
    grad = torch.zeros(case["rows"], case["width"], dtype=torch.float64, device="cuda")
    if order.numel():
        rows, counts = torch.unique_consecutive(at[order], return_counts=True)
        ends = torch.cumsum(counts, 0)
        for c in range(0, case["width"], 512):
            run_sum = torch.cumsum(state["grad_out"][order, c:c + 512].double(), 0)[ends - 1]
            run_sum[1:] -= run_sum[:-1].clone()
            grad[rows, c:c + 512] = run_sum * case["scale"]
    return grad


def _exact_loss(state, case):
    n = case["tokens"]
    x, w = state["hidden"].double(), state["weight"].double()
    losses = torch.zeros(n, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, dtype=torch.float64, device="cuda")
    step = case["op"] == "loss_step"
    dx = torch.zeros_like(x) if step else None
    dw = torch.zeros_like(w) if step else None
    for lo in range(0, n, 1024):
        part = slice(lo, min(n, lo + 1024))
        z = torch.mm(x[part], w.t())
        lse[part] = torch.logsumexp(z, dim=1)
        rows = torch.nonzero(state["targets"][part] != IGNORE)[:, 0]
        aim = state["targets"][part].long()[rows]
        losses[lo + rows] = lse[part][rows] - z[rows, aim]
        if step:
            share = torch.zeros_like(z)
            share[rows] = torch.softmax(z[rows], dim=1)
            share[rows, aim] -= 1.0
            share *= state["grad_losses"][part].double()[:, None]
            dx[part] = torch.mm(share, w)
            dw += torch.mm(share.t().contiguous(), x[part])
    return {"losses": losses, "lse": lse, "grad_hidden": dx, "grad_weight": dw} if step else {"losses": losses, "lse": lse}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("clip", "reduce_clip"):
        return _exact_clip(state, case | {"counts": state["counts"], "op_dtype": case["dtype"]})
    if op == "lookup":
        at = state["tokens"].long() - case["first"]
        out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        here = torch.nonzero((at >= 0) & (at < case["rows"]))[:, 0]
        out[here] = state["weight"][at[here]].double() * case["scale"]
        return out
    if op == "lookup_grad":
        return _exact_lookup_grad(state, case)
    return _exact_loss(state, case)
