"""Cases of the operators of a policy-gradient step around the gradient
all-reduce: the log probabilities of given tokens under a linear head, with the
entropy and the likeliest alternatives, their gradients, and the weights' update
by orthogonalised momentum (Newton-Schulz products), alone and as a whole step.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through ``ring_all_reduce_ar_amd``.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}
INDEX = {"i32": torch.int32, "i64": torch.int64}
IGNORE = -100
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # serving: the score of the token that one request has just sampled, with a few alternatives
        {"name": "log probs one bf16", "op": "log_probs", "tokens": 1, "vocab": 32_000, "width": 4096, "dtype": "bf16",
         "top": 5, "scale": 1.25, "ignored": 0.0, "index": "i64"},
        # serving: a small batch of requests, each with twenty alternatives
        {"name": "log probs few f16", "op": "log_probs", "tokens": 24, "vocab": 65_536, "width": 2048, "dtype": "f16",
         "top": 20, "scale": 1.0, "ignored": 0.0, "index": "i64"},
        # scoring a batch of prompts with alternatives
        {"name": "log probs batch bf16", "op": "log_probs", "tokens": 4096, "vocab": 65_536, "width": 2048,
         "dtype": "bf16", "top": 8, "scale": 1.0, "ignored": 0.05, "index": "i64"},
        # scores and entropies of a small fp32 model with odd sizes
        {"name": "log probs odd f32", "op": "log_probs", "tokens": 1021, "vocab": 32_003, "width": 770, "dtype": "f32",
         "top": 0, "scale": 0.75, "ignored": 0.1, "index": "i32"},
        # a policy-gradient step with an entropy bonus of that small model
        {"name": "policy step odd f32", "op": "policy_step", "tokens": 509, "vocab": 32_003, "width": 770,
         "dtype": "f32", "scale": 1.25, "entropy": True, "ignored": 0.1, "index": "i32"},
        # of a middling half-precision model
        {"name": "policy step f16", "op": "policy_step", "tokens": 2048, "vocab": 32_000, "width": 1024,
         "dtype": "f16", "scale": 1.0, "entropy": True, "ignored": 0.25, "index": "i64"},
        # of a large model's head
        {"name": "policy step large bf16", "op": "policy_step", "tokens": 6000, "vocab": 131_072, "width": 4096,
         "dtype": "bf16", "scale": 1.25, "entropy": True, "ignored": 0.02, "index": "i64"},
        # projections of a tiny model: latency counts
        {"name": "orthogonalize small f32", "op": "orthogonalize", "matrices": 4, "rows": 64, "cols": 192,
         "dtype": "f32"},
        # a few odd matrices, taller than wide
        {"name": "orthogonalize odd bf16", "op": "orthogonalize", "matrices": 3, "rows": 1027, "cols": 770,
         "dtype": "bf16"},
        # one wide matrix of a large model
        {"name": "orthogonalize large f32", "op": "orthogonalize", "matrices": 1, "rows": 4096, "cols": 8192,
         "dtype": "f32"},
        # the whole update of a small model's square matrices: bf16 gradients, fp32 weights
        {"name": "muon small bf16", "op": "muon", "ranks": 1, "matrices": 24, "rows": 256, "cols": 256,
         "dtype": "bf16", "weight_dtype": "f32", "nesterov": True},
        # of eight layers of a larger one, the weights' replicas of two ranks
        {"name": "muon layers bf16", "op": "muon", "ranks": 2, "matrices": 8, "rows": 2048, "cols": 4096,
         "dtype": "bf16", "weight_dtype": "bf16", "nesterov": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["log_probs", "policy_step", "orthogonalize", "muon"])
    if op in ("log_probs", "policy_step"):
        case = {"op": op, "tokens": _log_int(rng, 1, 6000), "vocab": _log_int(rng, 500, 131_072),
                "width": _log_int(rng, 64, 4096), "dtype": rng.choice(["f16", "bf16", "bf16", "f32"]),
                "scale": rng.choice([1.0, 0.75, 1.25, 1.5]), "ignored": rng.choice([0.0, 0.1, 0.5]),
                "index": rng.choice(["i32", "i64"])}
        if rng.random() < 0.7:
            case["width"] = max(64, case["width"] // 64 * 64)
        if case["dtype"] == "f32":
            case["width"] = min(case["width"], 1024)
        if op == "policy_step":
            return case | {"entropy": rng.random() < 0.7}
        return case | {"top": rng.choice([0, 0, 1, 3, 5, 8, 20, 20])}
    small, large = sorted((_log_int(rng, 16, 4096), _log_int(rng, 16, 8192)))
    small, large = min(small, 4096), max(small, large)
    room = 4096 * 4096 * (2 * 8192 + 4096)
    most = max(1, room // (small * small * (2 * large + small)))
    rows, cols = (small, large) if rng.random() < 0.6 else (large, small)
    case = {"op": op, "matrices": min(_log_int(rng, 1, 32), most), "rows": rows, "cols": cols,
            "dtype": rng.choice(["f32", "f16", "bf16", "bf16"])}
    if op == "muon":
        case |= {"ranks": rng.choice([1, 1, 2, 4]), "weight_dtype": rng.choice([case["dtype"], "f32"]),
                 "nesterov": rng.random() < 0.7}
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _on_grid(x, step, most):
    """Rounded to multiples of `step`, `most` of them at the most."""
    return (x / step).round_().clamp_(-most, most).mul_(step)


def _tokens(n, rows, g):
    """Token numbers as text has them: the k-th most frequent one about 1/k as
    often as the first, spread over the rows."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    k = (torch.exp(u * math.log(rows + 1.0)) - 1.0).long().clamp_(0, rows - 1)
    return (k * 7919 + 13) % rows


def _head(case, g):
    n, vocab, width, dt = case["tokens"], case["vocab"], case["width"], DTYPE[case["dtype"]]
    hidden = _normal(g, n, width)
    weight = _normal(g, vocab, width, std=1.5 / math.sqrt(width))
    if case.get("top"):
        # Alternatives are whole numbers, so their order must not hang on the
        # order of a sum: on these grids (as of weights kept in 7 bits) every
        # logit is a multiple of one step below 2^24 of them, exact in fp32.
        hidden = _on_grid(hidden, 0.125, 32)
        weight = _on_grid(weight, 2.0 ** round(math.log2(1.5 / math.sqrt(width) / 8)), 48)
    targets = _tokens(n, vocab, g)
    drop = torch.rand(n, generator=g, device="cuda") < case["ignored"]
    state = {"hidden": hidden.to(dt), "weight": weight.to(dt),
             "targets": torch.where(drop, torch.full_like(targets, IGNORE), targets).to(INDEX[case["index"]])}
    for name in ("log_probs", "entropy", "lse"):
        state[name] = torch.empty(n, device="cuda")
    if case["op"] == "log_probs":
        state["top_log_probs"] = torch.empty(n, case["top"], device="cuda")
        state["top_ids"] = torch.empty(n, case["top"], dtype=torch.int32, device="cuda")
    else:
        # of -mean(advantage * log p + 0.01 * entropy)
        state["grad_log_probs"] = _normal(g, n, std=1.0 / n)
        state["grad_entropy"] = torch.full((n,), -0.01 / n, device="cuda") if case["entropy"] else None
        state["grad_hidden"] = torch.empty_like(state["hidden"])
        state["grad_weight"] = torch.empty_like(state["weight"])
    return state


def _gradient(case, g, std):
    """A few directions that many tokens share, above noise of the same norm."""
    rows, cols = case["rows"], case["cols"]
    rank = min(8, rows, cols)
    x = _normal(g, rows, rank) @ _normal(g, rank, cols) * rank ** -0.5
    return (x + _normal(g, rows, cols)).mul_(std)


def _matrices(case, g):
    n, dt = case["matrices"], DTYPE[case["dtype"]]
    grads = [_gradient(case, g, 1e-3).to(dt) for _ in range(n)]
    if case["op"] == "orthogonalize":
        return {"grads": grads, "outs": [torch.empty_like(x) for x in grads]}
    wt = DTYPE[case["weight_dtype"]]
    momentum = [_gradient(case, g, 3e-4) for _ in range(n)]
    weights = [_normal(g, case["rows"], case["cols"], dtype=wt, std=case["cols"] ** -0.5) for _ in range(n)]
    return {"grads": grads, "momentum": momentum, "weights": weights,
            "momentum_out": [torch.empty_like(x) for x in momentum],
            "weights_out": [[torch.empty_like(x) for _ in range(case["ranks"])] for x in weights]}


def _update(case):
    """The hyperparameters of a step: the update as large as an Adam step's."""
    return {"decay": 0.95, "nesterov": case["nesterov"], "lr": 0.02, "weight_decay": 0.1,
            "update_scale": 0.2 * math.sqrt(max(case["rows"], case["cols"]))}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    head = case["op"] in ("log_probs", "policy_step")
    return {"case": case} | (_head(case, g) if head else _matrices(case, g))


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
    op, ready = case["op"], state.get("ready")
    if op in ("orthogonalize", "muon"):
        n, rows, cols = case["matrices"], case["rows"], case["cols"]
        if ready is None:
            import ring_all_reduce_ar_amd as ar
            ready = _comm(state, ar.ar_orthogonalize_workspace_bytes(n, rows, cols))
        ar, comm = ready
        if op == "orthogonalize":
            ar.ar_orthogonalize(comm, state["grads"], state["outs"], rows, cols, case["dtype"], steps=STEPS, eps=EPS)
            return state["outs"]
        ar.ar_muon_update(comm, state["grads"], state["momentum"], state["momentum_out"], state["weights"],
                          state["weights_out"], rows, cols, case["dtype"], case["weight_dtype"], steps=STEPS, eps=EPS,
                          **_update(case))
        return {"momentum": state["momentum_out"], "weights": state["weights_out"]}
    n, vocab, width, dtype = case["tokens"], case["vocab"], case["width"], case["dtype"]
    step, top = op == "policy_step", case.get("top", 0)
    if ready is None:
        import ring_all_reduce_ar_amd as ar
        ready = _comm(state, max(ar.ar_linear_log_probs_workspace_bytes(n, vocab, width, dtype, top=top),
                                 ar.ar_linear_log_probs_workspace_bytes(n, vocab, width, dtype, backward=True)
                                 if step else 0))
    ar, comm = ready
    ar.ar_linear_log_probs(comm, state["hidden"], state["weight"], state["targets"], state["log_probs"],
                           state["entropy"], state["lse"], n, vocab, width, dtype, top=top,
                           top_log_probs=state["top_log_probs"] if top else None,
                           top_ids=state["top_ids"] if top else None, scale=case["scale"], ignore_index=IGNORE)
    out = {"log_probs": state["log_probs"], "entropy": state["entropy"], "lse": state["lse"]}
    if not step:
        return out | {"top_log_probs": state["top_log_probs"], "top_ids": state["top_ids"]}
    ar.ar_linear_log_probs_backward(comm, state["hidden"], state["weight"], state["targets"], state["lse"],
                                    state["entropy"], state["grad_log_probs"], state["grad_entropy"],
                                    state["grad_hidden"], state["grad_weight"], n, vocab, width, dtype,
                                    scale=case["scale"], ignore_index=IGNORE)
    return out | {"grad_hidden": state["grad_hidden"], "grad_weight": state["grad_weight"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_head(state):
    case = state["case"]
    x, w = state["hidden"].float(), state["weight"].float()
    targets = state["targets"].long()
    kept = targets != IGNORE
    at = targets.clamp(min=0)[:, None]
    logits = (x @ w.t()) * case["scale"]
    peak = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - peak)
    total = e.sum(dim=1, keepdim=True)
    entropy = torch.log(total) - (e * (logits - peak)).sum(dim=1, keepdim=True) / total
    del e
    lse = peak + torch.log(total)
    log_probs = torch.where(kept, (logits.gather(1, at) - lse)[:, 0], torch.zeros((), device="cuda"))
    out = {"log_probs": log_probs, "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if case["op"] == "log_probs":
        values, ids = [], []
        for _ in range(case["top"]):  # the first of equal ones
            best = torch.argmax(logits, dim=1, keepdim=True)
            values.append(logits.gather(1, best) - lse)
            ids.append(best.int())
            logits.scatter_(1, best, float("-inf"))
        empty = torch.empty(case["tokens"], 0, device="cuda")
        return out | {"top_log_probs": torch.cat([empty] + values, 1), "top_ids": torch.cat([empty.int()] + ids, 1)}
    log_p = logits.sub_(lse)
    p = torch.exp(log_p)
    d = p * -(state["grad_log_probs"] * kept)[:, None]
    d.scatter_add_(1, at, (state["grad_log_probs"] * kept)[:, None])
    if case["entropy"]:
        d -= log_p.add_(entropy).mul_(p).mul_((state["grad_entropy"] * kept)[:, None])
    del p, log_p, logits
    d *= case["scale"]
    dt = DTYPE[case["dtype"]]
    return out | {"grad_hidden": (d @ w).to(dt), "grad_weight": (d.t() @ x).to(dt)}


def _plain_orthogonal(x):
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / x.square().sum().sqrt().clamp(min=EPS)
    a, b, c = QUINTIC
    for _ in range(STEPS):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if tall else x


def _plain_muon(state):
    case = state["case"]
    h = _update(case)
    decay, wt = h["decay"], DTYPE[case["weight_dtype"]]
    for grad, old, new, weight, replicas in zip(state["grads"], state["momentum"], state["momentum_out"],
                                                state["weights"], state["weights_out"]):
        grad = grad.float()
        new.copy_(decay * old + (1.0 - decay) * grad)
        update = decay * new + (1.0 - decay) * grad if h["nesterov"] else new
        update = _plain_orthogonal(update)
        weight = (weight.float() * (1.0 - h["lr"] * h["weight_decay"]) - h["lr"] * h["update_scale"] * update).to(wt)
        for replica in replicas:
            replica.copy_(weight)
    return {"momentum": state["momentum_out"], "weights": state["weights_out"]}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op in ("log_probs", "policy_step"):
        return _plain_head(state)
    if op == "orthogonalize":
        for x, out in zip(state["grads"], state["outs"]):
            out.copy_(_plain_orthogonal(x.float()))
        return state["outs"]
    return _plain_muon(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _orthogonal_flops(rows, cols):
    """Of one matrix: the iteration as it is written, or all steps but the last
    product on the small side's Gram matrix, whichever is less; half of every
    symmetric product is its mirror."""
    m, n = min(rows, cols), max(rows, cols)
    written = STEPS * (m * m * n + m ** 3 + 2 * m * m * n)
    gram = m * m * n + (4 * STEPS - 3) * m ** 3 + 2 * m * m * n
    return min(written, gram)


def work(case):
    op, e = case["op"], ESIZE[case["dtype"]]
    if op in ("log_probs", "policy_step"):
        n, vocab, width = case["tokens"], case["vocab"], case["width"]
        step = op == "policy_step"
        operands = (n + vocab) * width * e
        index = n * ESIZE["f32"] * (1 if case["index"] == "i32" else 2)
        small = n * (20 if step else 12 + 8 * case["top"])
        return {"bytes": operands * (2 if step else 1) + index + small,
                "flops": 2.0 * n * vocab * width * (3 if step else 1)}
    count = case["matrices"] * case["rows"] * case["cols"]
    flops = 1.0 * case["matrices"] * _orthogonal_flops(case["rows"], case["cols"])
    if op == "orthogonalize":
        return {"bytes": 2 * count * e, "flops": flops}
    return {"bytes": count * (e + 8 + (1 + case["ranks"]) * ESIZE[case["weight_dtype"]]), "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_head(state, case):
    n, vocab = case["tokens"], case["vocab"]
    x, w = state["hidden"].double(), state["weight"].double()
    step, top = case["op"] == "policy_step", case.get("top", 0)
    out = {k: torch.zeros(n, dtype=torch.float64, device="cuda") for k in ("log_probs", "entropy", "lse")}
    if step:
        out |= {"grad_hidden": torch.zeros_like(x), "grad_weight": torch.zeros_like(w)}
    else:
        out |= {"top_log_probs": torch.zeros(n, top, dtype=torch.float64, device="cuda"),
                "top_ids": torch.zeros(n, top, dtype=torch.int32, device="cuda")}
    for lo in range(0, n, 512):
        part = slice(lo, min(n, lo + 512))
        log_p = torch.log_softmax(torch.mm(x[part], w.t()) * case["scale"], dim=1)
        p = torch.exp(log_p)
        aim = state["targets"][part].long()
        rows = torch.nonzero(aim != IGNORE)[:, 0]
        out["lse"][part] = torch.logsumexp(torch.mm(x[part], w.t()) * case["scale"], dim=1)
        out["entropy"][part] = -(p * log_p).sum(1)
        out["log_probs"][lo + rows] = log_p[rows, aim[rows]]
        if top:
            best, ids = torch.sort(log_p, dim=1, descending=True, stable=True)
            out["top_log_probs"][part], out["top_ids"][part] = best[:, :top], ids[:, :top].int()
        if step:
            d = torch.zeros_like(log_p)
            gain = state["grad_log_probs"][part].double()[rows]
            d[rows] = -p[rows] * gain[:, None]
            d[rows, aim[rows]] += gain
            if case["entropy"]:
                bonus = state["grad_entropy"][part].double()[rows]
                d[rows] -= p[rows] * (log_p[rows] + out["entropy"][part][rows][:, None]) * bonus[:, None]
            d *= case["scale"]
            out["grad_hidden"][part] = torch.mm(d, w)
            out["grad_weight"] += torch.mm(d.t().contiguous(), x[part])
    return out


def _exact_orthogonal(x):
    """The same polynomial as a product P x, by its factors on the Gram matrix."""
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    x = x / max(float(torch.linalg.matrix_norm(x)), EPS)
    gram = torch.mm(x, x.t())
    eye = torch.eye(gram.shape[0], dtype=torch.float64, device="cuda")
    product = eye
    for _ in range(STEPS):
        factor = QUINTIC[0] * eye + torch.mm(QUINTIC[1] * eye + QUINTIC[2] * gram, gram)
        product = torch.mm(factor, product)
        gram = torch.mm(torch.mm(factor, gram), factor)
    x = torch.mm(product, x)
    return x.t() if tall else x


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("log_probs", "policy_step"):
        return _exact_head(state, case)
    if case["op"] == "orthogonalize":
        return [_exact_orthogonal(x.double()) for x in state["grads"]]
    h = _update(case)
    out = {"momentum": [], "weights": []}
    for grad, old, weight in zip(state["grads"], state["momentum"], state["weights"]):
        grad = grad.double()
        new = torch.lerp(grad, old.double(), h["decay"])
        update = _exact_orthogonal(torch.lerp(grad, new, h["decay"]) if h["nesterov"] else new)
        weight = weight.double()
        weight = weight - h["lr"] * (h["weight_decay"] * weight + h["update_scale"] * update)
        out["momentum"].append(new)
        out["weights"].append([weight] * case["ranks"])
    return out
