"""Timed cases of the operators around an expert block in a training step.

Three operators, each with its gradient: the router's balance loss with the per-expert counts, the norms before and
after a block fused with its gate and residual scale, and distillation from a teacher's top logits. A case names an
operator, a direction and sizes; `run` makes one pass, either in a plain form written out in torch operations in 32
bits or, where `own` is true, through the package's entry points.
"""
import math

import torch

own = False  # set from outside: False runs the plain form, True the package's kernels

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases

def _balance(direction, tokens, experts, topk, dtype, score="softmax", groups=0, masked=False, **more):
    """groups = 0: one group without offsets; otherwise that many packed sequences of uneven lengths."""
    return dict(more, op="balance", direction=direction, tokens=tokens, experts=experts, topk=topk, dtype=dtype,
                score=score, groups=groups, masked=masked)


def _norm(direction, tokens, width, dtype, gate="channel", res_scale=1.0, **more):
    return dict(more, op="norm", direction=direction, tokens=tokens, width=width, dtype=dtype, gate=gate,
                res_scale=res_scale)


def _distill(direction, rows, vocab, topk, dtype, tau=1.0, tail=False, pad=0, **more):
    """pad: unused columns after each row's vocabulary (a vocabulary padded to a round width)."""
    return dict(more, op="distill", direction=direction, rows=rows, vocab=vocab, topk=topk, dtype=dtype, tau=tau,
                tail=tail, pad=pad)


def listed():
    return [
        # the aux loss's full workload: every token of a training step's router
        _balance("forward", 65536, 128, 8, "fp32", name="balance fwd 65536x128 fp32"),
        # its gradient, with the router's logits kept in 16 bits
        _balance("backward", 65536, 128, 8, "bf16", name="balance bwd 65536x128 bf16"),
        # a small microbatch with few experts: the call's latency
        _balance("forward", 257, 8, 2, "fp32", name="balance fwd 257x8 fp32"),
        # packed sequences, each with its own loss, prompts masked out, normalised sigmoid scores
        _balance("forward", 30011, 60, 6, "bf16", score="sigmoid", groups=16, masked=True,
                 name="balance fwd 30011x60 bf16 packed"),
        # the boundary between two blocks of a training step, a learned scale a channel
        _norm("forward", 16384, 4096, "bf16", name="norm fwd 16384x4096 bf16"),
        _norm("backward", 16384, 4096, "bf16", name="norm bwd 16384x4096 bf16"),
        # one token while answering: latency
        _norm("forward", 1, 2048, "bf16", name="norm fwd 1x2048 bf16"),
        # 32-bit training at a small odd-sized batch, a gate a token (a shared expert's) and a scaled residual
        _norm("backward", 3001, 1000, "fp32", gate="token", res_scale=0.8, name="norm bwd 3001x1000 fp32"),
        # a training step's loss and gradient together over a large vocabulary, with the teacher's remaining mass
        _distill("both", 4096, 131072, 64, "bf16", tau=2.0, tail=True, name="distill both 4096x131072 bf16"),
        # the loss alone, on held-out data
        _distill("forward", 2048, 32768, 128, "fp32", name="distill fwd 2048x32768 fp32"),
        # few rows: the end of a ragged batch
        _distill("both", 16, 65536, 20, "bf16", name="distill both 16x65536 bf16"),
        # the gradient alone, an odd vocabulary inside rows of a round width
        _distill("backward", 1021, 50001, 50, "bf16", tau=1.5, pad=47, name="distill bwd 1021x50001 bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["balance", "norm", "distill"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "balance":
        experts = rng.choice([8, 16, 32, 64, 128, 256, _log_int(rng, 4, 512)])
        tokens = _log_int(rng, 64, 1 << 17)
        return _balance(rng.choice(["forward", "backward"]), tokens, experts, min(experts, rng.choice([1, 2, 4, 6, 8])),
                        dtype, score=rng.choice(["softmax", "sigmoid"]),
                        groups=rng.choice([0, 0, _log_int(rng, 1, 64)]), masked=rng.random() < 0.5)
    if op == "norm":
        width = rng.choice([512, 1024, 2048, 4096, 8192, 8 * _log_int(rng, 8, 1024), _log_int(rng, 65, 5000)])
        tokens = _log_int(rng, 1, min(32768, (1 << 26) // width))
        return _norm(rng.choice(["forward", "backward"]), tokens, width, dtype, gate=rng.choice(["channel", "token", "none"]),
                     res_scale=rng.choice([1.0, round(rng.uniform(0.3, 1.5), 3)]))
    vocab = rng.choice([32768, 65536, 131072, _log_int(rng, 1000, 160000)])
    rows = _log_int(rng, 1, min(8192, (1 << 27) // vocab))
    return _distill(rng.choice(["forward", "backward", "both"]), rows, vocab, rng.choice([8, 20, 50, 64, 100, 128]), dtype,
                    tau=rng.choice([1.0, round(rng.uniform(0.5, 4.0), 2)]), tail=rng.random() < 0.5,
                    pad=rng.choice([0, 0, rng.randrange(1, 64)]))


# ------------------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    state = {"balance": _prepare_balance, "norm": _prepare_norm, "distill": _prepare_distill}[case["op"]](case, g)
    return dict(state, case=dict(case))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _prepare_balance(case, g):
    N, E, K, dt = case["tokens"], case["experts"], case["topk"], DTYPES[case["dtype"]]
    # a router prefers some experts over others: a bias an expert, then the tokens' own spread
    logits = (1.5 * _randn(g, N, E) + _randn(g, E)).to(dt)
    ids = logits.float().topk(K, dim=1).indices.to(torch.int32)
    ids[_rand(g, N, K) < 0.02] = -1  # dropped by the experts' capacity
    mask = offs = None
    if case["masked"]:
        mask = (_rand(g, N) > 0.15).to(torch.uint8)
    if case["groups"]:
        cuts = torch.sort((_rand(g, case["groups"] - 1) * (N + 1)).to(torch.int64)).values
        offs = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts,
                          torch.full((1,), N, dtype=torch.int64, device="cuda")])
    state = {"logits": logits, "ids": ids, "mask": mask, "offs": offs, "coeff": 0.01}
    if case["direction"] == "backward":  # what the forward pass left behind
        state["counts"], state["tokens"] = _counts(ids, mask, offs, N, E)
        state["dloss"] = 0.5 + _rand(g, 1)
    return state


def _prepare_norm(case, g):
    T, H, dt = case["tokens"], case["width"], DTYPES[case["dtype"]]
    state = {"y": (0.7 * _randn(g, T, H)).to(dt), "w_post": (1 + 0.2 * _randn(g, H)).to(dt),
             "w_pre": (1 + 0.2 * _randn(g, H)).to(dt), "eps": 1e-6, "res_scale": case["res_scale"], "gate": None}
    if case["gate"] == "channel":
        state["gate"] = (0.5 + 0.2 * _randn(g, H)).to(dt)
    elif case["gate"] == "token":
        state["gate"] = _rand(g, T, 1).to(dt)
    if case["direction"] == "forward":
        state["x"] = (2.0 * _randn(g, T, H)).to(dt)
    else:
        state["h"] = (2.0 * _randn(g, T, H)).to(dt)  # the residual stream behind the block
        state["dh"] = (0.01 * _randn(g, T, H)).to(dt)
        state["du"] = (0.01 * _randn(g, T, H)).to(dt)
    return state


def _prepare_distill(case, g):
    T, V, K, dt = case["rows"], case["vocab"], case["topk"], DTYPES[case["dtype"]]
    K = min(K, V)
    buf = torch.zeros(T, V + case["pad"], dtype=dt, device="cuda")
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    teacher = torch.empty(T, K, device="cuda")
    lse = torch.empty(T, device="cuda") if case["tail"] else None
    step = max(1, (1 << 27) // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        z = 2.0 * _randn(g, b - a, V)
        t = 0.8 * z + 1.2 * _randn(g, b - a, V)  # a teacher whose view the student partly shares
        top = t.topk(K, dim=1)
        # few tokens are likely: a head that falls off over the list, half of it known to the student
        head = (5 + 5 * case["tau"]) * torch.exp(-torch.arange(K, device="cuda") / 12)
        t.scatter_(1, top.indices, top.values + head)
        z.scatter_add_(1, top.indices, (0.5 * head).expand(b - a, K))
        buf[a:b, :V] = z.to(dt)
        teacher[a:b], ids[a:b] = top.values + head, top.indices.to(torch.int32)
        if lse is not None:
            lse[a:b] = torch.logsumexp(t / case["tau"], dim=1)
        del z, t, top
    # lists are cut at a cumulated mass, so some are shorter than K; prompts carry no weight
    length = 1 + (_rand(g, T, 1) * 2 * K).to(torch.int32)
    ids[torch.arange(K, device="cuda")[None, :] >= length] = -1
    weights = (_rand(g, T) > 0.1).float()
    weights[0] = 1.0
    return {"logits": buf[:, :V], "ids": ids, "teacher": teacher, "teacher_lse": lse, "weights": weights,
            "tau": case["tau"], "scale": 1.0 / T}


# ------------------------------------------------------------------------------------------------------------ passes

def run(state):
    case = state["case"]
    if own:
        return {"balance": _own_balance, "norm": _own_norm, "distill": _own_distill}[case["op"]](state, case["direction"])
    return {"balance": _plain_balance, "norm": _plain_norm, "distill": _plain_distill}[case["op"]](state, case["direction"])


# The package's entry points, with the outputs and workspaces that a training loop keeps from step to step.

def _own_balance(s, direction):
    import deterministic_gradient_reduction_gb300 as dgr
    x, score = s["logits"], s["case"]["score"]
    N, E = x.shape
    G = 1 if s["offs"] is None else s["offs"].numel() - 1
    if direction == "forward":
        if "ws" not in s:
            s["ws"] = dgr.workspace(dgr.router_balance_workspace_bytes(N, E, G))
            s["out"] = (torch.empty(1, device="cuda"), torch.empty(G, E, dtype=torch.int32, device="cuda"),
                        torch.empty(G, dtype=torch.int32, device="cuda"))
        loss, counts, tokens = dgr.router_balance(x, s["ids"], s["coeff"], offs=s["offs"], mask=s["mask"], score=score,
                                                  loss=s["out"][0], counts=s["out"][1], tokens=s["out"][2], ws=s["ws"])
        return {"loss": loss, "counts": counts, "tokens": tokens}
    if "out" not in s:
        s["out"] = torch.empty_like(x)
    return {"dlogits": dgr.router_balance_backward(x, s["counts"], s["tokens"], s["ids"].shape[1], s["coeff"],
                                                   offs=s["offs"], mask=s["mask"], score=score, dloss=s["dloss"],
                                                   dlogits=s["out"])}


def _own_norm(s, direction):
    import deterministic_gradient_reduction_gb300 as dgr
    y, gate = s["y"], s["gate"]
    T, H = y.shape
    if direction == "forward":
        if "out" not in s:
            s["out"] = (torch.empty_like(y), torch.empty_like(y))
        h, u = dgr.block_norm(s["x"], y, w_post=s["w_post"], gate=gate, res_scale=s["res_scale"], w_pre=s["w_pre"],
                              eps=s["eps"], h=s["out"][0], u=s["out"][1])
        return {"h": h, "u": u}
    if "ws" not in s:
        s["ws"] = dgr.workspace(dgr.block_norm_workspace_bytes(T, H))
        w = lambda: torch.empty(H, device="cuda")  # noqa: E731
        s["out"] = {"dx": torch.empty_like(y), "dy": torch.empty_like(y), "dw_post": w(), "dw_pre": w()}
        if gate is not None:
            s["out"]["dgate"] = w() if gate.dim() == 1 else torch.empty(T, 1, device="cuda")
    return dgr.block_norm_backward(s["h"], y, s["dh"], s["du"], w_post=s["w_post"], gate=gate, res_scale=s["res_scale"],
                                   w_pre=s["w_pre"], eps=s["eps"], ws=s["ws"], **s["out"])


def _own_distill(s, direction):
    import deterministic_gradient_reduction_gb300 as dgr
    z = s["logits"]
    T, V = z.shape
    if "ws" not in s:
        s["ws"] = dgr.workspace(dgr.topk_distill_workspace_bytes(T))
        s["out"] = {"loss": torch.empty(1, device="cuda"), "row_loss": torch.empty(T, device="cuda"),
                    "dlogits": torch.empty(T, V, dtype=z.dtype, device="cuda") if direction != "forward" else None}
    o = s["out"]
    same = dict(tau=s["tau"], teacher_lse=s["teacher_lse"], weights=s["weights"], scale=s["scale"], ws=s["ws"])
    if direction == "backward":
        return {"dlogits": dgr.topk_distill_backward(z, s["ids"], s["teacher"], dlogits=o["dlogits"], **same)}
    loss, rows = dgr.topk_distill(z, s["ids"], s["teacher"], loss=o["loss"], row_loss=o["row_loss"], dlogits=o["dlogits"],
                                  **same)
    return {"loss": loss, "row_loss": rows, "dlogits": o["dlogits"]}


# The plain forms: torch operations in 32 bits, rounded once at the end.

def _group_of(offs, N):
    """Each token's group."""
    if offs is None:
        return torch.zeros(N, dtype=torch.int64, device="cuda")
    at = torch.arange(N, device="cuda")
    return (at[:, None] >= offs[None, 1:-1]).sum(1)


def _counts(ids, mask, offs, N, E):
    G = 1 if offs is None else offs.numel() - 1
    group = _group_of(offs, N)
    live = torch.ones(N, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    tokens = torch.zeros(G, dtype=torch.int32, device="cuda").index_add_(0, group, live.to(torch.int32))
    takes = (ids >= 0) & live[:, None]
    slot = torch.where(takes, group[:, None] * E + ids, G * E)
    counts = torch.zeros(G * E + 1, dtype=torch.int32, device="cuda")
    counts.index_add_(0, slot.reshape(-1).to(torch.int64), torch.ones(slot.numel(), dtype=torch.int32, device="cuda"))
    return counts[:-1].reshape(G, E), tokens


def _scores(logits, score):
    x = logits.float()
    if score == "sigmoid":
        sig = 1 / (1 + torch.exp(-x))
        return sig / sig.sum(1, keepdim=True), sig
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True), None


def _plain_balance(s, direction):
    x, offs, mask = s["logits"], s["offs"], s["mask"]
    N, E = x.shape
    G = 1 if offs is None else offs.numel() - 1
    K = s["ids"].shape[1]
    p, sig = _scores(x, s["case"]["score"])
    group = _group_of(offs, N)
    live = torch.ones(N, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    if direction == "forward":
        counts, tokens = _counts(s["ids"], mask, offs, N, E)
        n = tokens.float().clamp(min=1)
        member = ((group[None, :] == torch.arange(G, device="cuda")[:, None]) & live[None, :]).float()
        mass = member @ p if G > 1 else (p * live[:, None]).sum(0, keepdim=True)
        per = (counts.float() * mass).sum(1) / (n * n)
        return {"loss": (s["coeff"] * E / (G * K) * per.sum()).reshape(1), "counts": counts, "tokens": tokens}
    n = s["tokens"].float().clamp(min=1)
    a = s["dloss"] * s["coeff"] * E / (G * K) * s["counts"].float() / (n * n)[:, None]
    a = a[group]
    d = p * (a - (a * p).sum(1, keepdim=True))
    if sig is not None:
        d = d * (1 - sig)
    return {"dlogits": torch.where(live[:, None], d, torch.zeros_like(d)).to(x.dtype)}


def _plain_norm(s, direction):
    y, w1, w2 = s["y"].float(), s["w_post"].float(), s["w_pre"].float()
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    alpha, eps, dt = s["res_scale"], s["eps"], s["y"].dtype
    r1 = torch.rsqrt((y * y).mean(1, keepdim=True) + eps)
    if direction == "forward":
        h = alpha * s["x"].float() + gate * (y * r1 * w1)
        r2 = torch.rsqrt((h * h).mean(1, keepdim=True) + eps)
        return {"h": h.to(dt), "u": (h * r2 * w2).to(dt)}
    h, dh, du = s["h"].float(), s["dh"].float(), s["du"].float()
    r2 = torch.rsqrt((h * h).mean(1, keepdim=True) + eps)
    hh = h * r2
    v = du * w2
    D = dh + r2 * (v - hh * (v * hh).mean(1, keepdim=True))
    yy = y * r1
    q = gate * D * w1
    out = {"dx": (alpha * D).to(dt), "dy": (r1 * (q - yy * (q * yy).mean(1, keepdim=True))).to(dt),
           "dw_post": (gate * D * yy).sum(0), "dw_pre": (du * hh).sum(0)}
    if s["gate"] is not None:
        n = D * yy * w1
        out["dgate"] = n.sum(0) if s["gate"].dim() == 1 else n.sum(1, keepdim=True)
    return out


def _plain_distill(s, direction):
    z, ids = s["logits"], s["ids"].to(torch.int64)
    T, V = z.shape
    valid = ids >= 0
    at = torch.where(valid, ids, 0)
    x = z.float() * (1.0 / s["tau"])
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    t = torch.where(valid, s["teacher"] * (1.0 / s["tau"]), -math.inf)
    if s["teacher_lse"] is None:
        log_q = t - t.amax(1, keepdim=True)
        log_q = log_q - torch.log(torch.exp(log_q).sum(1, keepdim=True))
    else:
        log_q = t - s["teacher_lse"][:, None]
    q = torch.exp(log_q)
    log_p = x.gather(1, at) - m - torch.log(total)
    live = (s["weights"] != 0) & valid.any(1)
    rows = torch.where(q > 0, q * (log_q - log_p), 0.0).sum(1)
    if s["teacher_lse"] is not None:
        q_rest = (1 - q.sum(1, keepdim=True)).clamp(min=0)
        slot = torch.where(valid, ids, V)
        outside = torch.ones(T, V + 1, dtype=torch.bool, device="cuda").scatter_(1, slot, False)[:, :V]
        p_rest = torch.where(outside, e, 0.0).sum(1, keepdim=True) / total
        rest = torch.where(q_rest > 0, q_rest * (torch.log(q_rest) - torch.log(p_rest)), 0.0)
        rows = rows + rest[:, 0]
    rows = torch.where(live, rows, 0.0)
    out = {}
    if direction != "backward":
        out = {"loss": (s["scale"] * (s["weights"] * rows).sum()).reshape(1), "row_loss": rows}
    if direction != "forward":
        d = e / total
        if s["teacher_lse"] is not None:
            d = torch.where(outside, d * (1 - q_rest / p_rest), d)
        d.scatter_add_(1, at, torch.where(valid, -q, 0.0))
        factor = torch.where(live, s["weights"] * (s["scale"] / s["tau"]), 0.0)
        out["dlogits"] = (d * factor[:, None]).to(z.dtype)
    return out


# ------------------------------------------------------------------------------------------------------ work, 64 bits

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "balance":
        N, E, K, G = case["tokens"], case["experts"], case["topk"], max(1, case["groups"])
        side = N * (1 if case["masked"] else 0) + 8 * (G + 1) + 4 * G * (E + 1)
        if case["direction"] == "forward":
            return {"bytes": N * (E * es + 4 * K) + side + 4, "flops": 6 * N * E}
        return {"bytes": 2 * N * E * es + side + 4, "flops": 9 * N * E}
    if case["op"] == "norm":
        T, H = case["tokens"], case["width"]
        gate = {"channel": H, "token": T, "none": 0}[case["gate"]]
        if case["direction"] == "forward":
            return {"bytes": (4 * T * H + 2 * H + gate) * es, "flops": 10 * T * H}
        return {"bytes": (6 * T * H + 2 * H + gate) * es + 4 * (2 * H + gate), "flops": 26 * T * H}
    T, V, K = case["rows"], case["vocab"], case["topk"]
    lists = T * (8 * K + 4 + (4 if case["tail"] else 0))
    grad = case["direction"] != "forward"
    loss = 4 * T + 4 if case["direction"] != "backward" else 0
    return {"bytes": T * V * es * (2 if grad else 1) + lists + loss, "flops": (7 if grad else 4) * T * V}


def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "norm": _exact_norm, "distill": _exact_distill}[case["op"]](s, case)


def _exact_balance(s, case):
    """Group by group from the definition; the gradient as the softmax's Jacobian applied to the counts."""
    x = s["logits"].double()
    N, E = x.shape
    K = case["topk"]
    if case["score"] == "sigmoid":
        x = torch.nn.functional.logsigmoid(x)
    p = torch.softmax(x, dim=1)
    offs = [0, N] if s["offs"] is None else s["offs"].tolist()
    live = torch.ones(N, dtype=torch.float64, device="cuda") if s["mask"] is None else s["mask"].double()
    G = len(offs) - 1
    loss, grad = 0.0, torch.zeros_like(p)
    for g in range(G):
        a, b = offs[g], offs[g + 1]
        n = float(live[a:b].sum())
        if n == 0:
            continue
        picked = s["ids"][a:b][live[a:b] > 0].reshape(-1)
        c = torch.bincount(picked[picked >= 0].long(), minlength=E).double()
        share, mean = c / (n * K), (p[a:b] * live[a:b, None]).sum(0) / n
        loss += s["coeff"] * E / G * float((share * mean).sum())
        up = s["coeff"] * E / G * share / n
        inner = p[a:b] @ up
        grad[a:b] = live[a:b, None] * (p[a:b] * up[None, :] - p[a:b] * inner[:, None])
    if case["direction"] == "forward":
        return {"loss": torch.tensor([loss], dtype=torch.float64), "counts": None, "tokens": None}
    if case["score"] == "sigmoid":
        grad = grad * torch.sigmoid(-s["logits"].double())
    return {"dlogits": grad * s["dloss"].double()}


def _exact_norm(s, case):
    """In slices of rows, the norms' Jacobians applied as products of whole rows."""
    T, H = s["y"].shape
    f = lambda t: t.double()  # noqa: E731
    w1, w2, eps, alpha = f(s["w_post"]), f(s["w_pre"]), s["eps"], float(s["res_scale"])
    gate = None if s["gate"] is None else f(s["gate"])
    parts, sums = [], {}
    step = max(1, (1 << 25) // H)

    def scale_of(v):
        return 1.0 / torch.sqrt(v.pow(2).sum(1) / H + eps)

    for a in range(0, T, step):
        rows = slice(a, min(T, a + step))
        y = f(s["y"][rows])
        g = 1.0 if gate is None else gate[None, :] if gate.dim() == 1 else gate[rows]
        k1 = scale_of(y)[:, None]
        normed = y * k1
        if case["direction"] == "forward":
            h = f(s["x"][rows]) * alpha + normed * w1 * g
            parts.append({"h": h, "u": h * scale_of(h)[:, None] * w2})
            continue
        h, du = f(s["h"][rows]), f(s["du"][rows])
        k2 = scale_of(h)[:, None]
        top = du * w2
        D = f(s["dh"][rows]) + top * k2 - h * ((top * h).sum(1, keepdim=True) * k2 ** 3 / H)
        q = D * w1 * g
        got = {"dx": D * alpha, "dy": q * k1 - y * ((q * y).sum(1, keepdim=True) * k1 ** 3 / H)}
        add = {"dw_post": (D * g * normed).sum(0), "dw_pre": (du * h * k2).sum(0)}
        if gate is not None and gate.dim() == 1:
            add["dgate"] = (D * normed * w1).sum(0)
        elif gate is not None:
            got["dgate"] = (D * normed * w1).sum(1, keepdim=True)
        for k, v in add.items():
            sums[k] = sums.get(k, 0.0) + v
        parts.append(got)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return {**out, **sums}


def _exact_distill(s, case):
    """In slices of rows: log-probabilities by logsumexp, the gradient as the mass of the student less the target's."""
    T, V = s["logits"].shape
    tau = float(case["tau"])
    rows_out, grads = [], []
    step = max(1, (1 << 26) // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        lp = s["logits"][a:b].double() / tau
        lp = lp - torch.logsumexp(lp, dim=1, keepdim=True)
        ids = s["ids"][a:b].long()
        valid = ids >= 0
        t = (s["teacher"][a:b].double() / tau).masked_fill(~valid, -math.inf)
        lq = t - (torch.logsumexp(t, 1, keepdim=True) if s["teacher_lse"] is None else s["teacher_lse"][a:b, None].double())
        q = torch.exp(lq).masked_fill(~valid, 0.0)
        take = ids.clamp(min=0)
        got = (torch.special.xlogy(q, q) - q * lp.gather(1, take).masked_fill(~valid, 0.0)).sum(1)
        target = torch.zeros(b - a, V, dtype=torch.float64, device="cuda").scatter_add_(1, take, q)
        if s["teacher_lse"] is not None:
            left = (1 - q.sum(1)).clamp(min=0)
            inside = torch.zeros(b - a, V, dtype=torch.bool, device="cuda")
            inside[torch.nonzero(valid)[:, 0], ids[valid]] = True
            l_rest = torch.logsumexp(lp.masked_fill(inside, -math.inf), 1)
            got = got + torch.special.xlogy(left, left) - left * l_rest
            target = target + torch.where(inside, 0.0, torch.exp(lp - l_rest[:, None]) * left[:, None])
        live = ((s["weights"][a:b] != 0) & valid.any(1)).double()
        rows_out.append(got * live)
        if case["direction"] != "forward":
            k = live * s["weights"][a:b].double() * (s["scale"] / tau)
            grads.append(((torch.exp(lp) - target) * k[:, None]).to(torch.float64 if T * V < 1 << 27 else torch.float32))
        del lp, target
    out = {}
    if case["direction"] != "backward":
        r = torch.cat(rows_out)
        out = {"loss": (r * s["weights"].double()).sum().reshape(1) * s["scale"], "row_loss": r}
    if case["direction"] != "forward":
        out["dlogits"] = torch.cat(grads)
    return out
