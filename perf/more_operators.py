"""Timed cases of three more operators of a training step, each with its gradient.

The gated feed-forward of grouped experts (both projections, the activation and the product), the norm of queries and
keys for each head with their rotation by position, and the log probabilities of given tokens with the entropy and the
top alternatives. A case names an operator, a direction and sizes; `run` makes one pass, either in a plain form written
out in torch operations in 32 bits or, where `own` is true, through the package's entry points.
"""
import math

import torch

own = False  # set from outside: False runs the plain form, True the package's kernels

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------------- cases

def _ffn(direction, tokens, width, hidden, experts, act="silu", keep=False, **more):
    """tokens: rows over all experts; keep: the forward pass leaves the pre-activations for its gradient."""
    return dict(more, op="ffn", direction=direction, tokens=tokens, width=width, hidden=hidden, experts=experts, act=act,
                keep=keep)


def _qk(direction, tokens, heads, kv_heads, dim, dtype, rotary=0, interleaved=False, **more):
    """rotary: how many of a head's elements are rotated (0: all)."""
    return dict(more, op="qk", direction=direction, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                rotary=rotary or dim, interleaved=interleaved)


def _logp(direction, rows, vocab, dtype, top=0, tau=1.0, pad=0, **more):
    """top: how many alternatives a row gives; pad: unused columns after each row's vocabulary."""
    return dict(more, op="logp", direction=direction, rows=rows, vocab=vocab, dtype=dtype, top=top, tau=tau, pad=pad)


def listed():
    return [
        # a training step's experts, at the sizes of the grouped weight gradient's workload
        _ffn("forward", 32768, 2048, 4096, 8, keep=True, name="ffn fwd 32768x2048x4096 E8"),
        # their gradient, to the pre-activations and to the tokens
        _ffn("backward", 32768, 2048, 4096, 8, name="ffn bwd 32768x2048x4096 E8"),
        # one token while answering: the weights' reading
        _ffn("forward", 1, 4096, 8192, 1, name="ffn fwd 1x4096x8192"),
        # a small batch over many experts, odd sizes, no expert's rows a whole tile
        _ffn("forward", 1021, 1000, 1416, 24, act="gelu", keep=True, name="ffn fwd 1021x1000x1416 E24"),
        # the queries and keys of a training step, grouped heads, cut out of one packed projection
        _qk("forward", 16384, 32, 8, 128, "bf16", name="qk fwd 16384x32+8x128 bf16"),
        _qk("backward", 16384, 32, 8, 128, "bf16", name="qk bwd 16384x32+8x128 bf16"),
        # one token while answering: latency
        _qk("forward", 1, 32, 8, 128, "bf16", name="qk fwd 1x32+8x128 bf16"),
        # 32-bit training at a small odd-sized batch, half of a head's elements rotated, neighbours paired
        _qk("backward", 3001, 12, 4, 80, "fp32", rotary=40, interleaved=True, name="qk bwd 3001x12+4x80 fp32"),
        # scores of sampled tokens in a policy's training step, and their gradient with the entropy's
        _logp("forward", 4096, 131072, "bf16", name="logp fwd 4096x131072 bf16"),
        _logp("backward", 4096, 131072, "bf16", name="logp bwd 4096x131072 bf16"),
        # a teacher's lists for distillation: an odd vocabulary inside rows of a round width
        _logp("forward", 2048, 50001, "fp32", top=64, tau=2.0, pad=47, name="logp fwd 2048x50001 fp32 top 64"),
        # one token while answering, with the alternatives that a user asked for
        _logp("forward", 1, 65536, "bf16", top=20, name="logp fwd 1x65536 bf16 top 20"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["ffn", "qk", "logp"])
    if op == "ffn":
        width = rng.choice([512, 1024, 2048, 4096, 8 * _log_int(rng, 8, 640)])
        hidden = rng.choice([512, 1024, 2048, 4096, 8192, 8 * _log_int(rng, 8, 1024)])
        experts = min(rng.choice([1, 1, 8, 16, 60, 128, _log_int(rng, 2, 128)]), max(1, (1 << 28) // (width * hidden)))
        tokens = _log_int(rng, 1, min(32768, (1 << 38) // (width * hidden)))
        direction = rng.choice(["forward", "backward"])
        return _ffn(direction, tokens, width, hidden, experts, act=rng.choice(["silu", "gelu"]),
                    keep=direction == "forward" and rng.random() < 0.5)
    dtype = rng.choice(["bf16", "fp32"])
    if op == "qk":
        dim = rng.choice([64, 128, 128, 256, 2 * _log_int(rng, 8, 128)])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        tokens = _log_int(rng, 1, min(32768, (1 << 26) // ((heads + kv) * dim)))
        return _qk(rng.choice(["forward", "backward"]), tokens, heads, kv, dim, dtype,
                   rotary=rng.choice([dim, dim, 2 * max(1, dim // 4)]), interleaved=rng.random() < 0.3)
    vocab = rng.choice([32768, 65536, 131072, _log_int(rng, 1000, 160000)])
    rows = _log_int(rng, 1, min(8192, (1 << 28) // vocab))
    direction = rng.choice(["forward", "forward", "backward"])
    return _logp(direction, rows, vocab, dtype, top=rng.choice([0, 1, 5, 20, 64]) if direction == "forward" else 0,
                 tau=rng.choice([1.0, round(rng.uniform(0.5, 2.0), 2)]), pad=rng.choice([0, 0, rng.randrange(1, 64)]))


# ------------------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    state = {"ffn": _prepare_ffn, "qk": _prepare_qk, "logp": _prepare_logp}[case["op"]](case, g, int(seed))
    return dict(state, case=dict(case))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _prepare_ffn(case, g, seed):
    T, H, F, E = case["tokens"], case["width"], case["hidden"], case["experts"]
    h = torch.Generator().manual_seed(seed)  # how many rows each expert has: a host's plan would know it too
    share = torch.exp(0.4 * torch.randn(E, generator=h, dtype=torch.float64))
    count = torch.bincount(torch.multinomial(share, T, replacement=True, generator=h), minlength=E)
    offs = torch.zeros(E + 1, dtype=torch.int64)
    offs[1:] = count.cumsum(0)
    bf = torch.bfloat16
    s = {"w_gate": (H ** -0.5 * _randn(g, E, F, H)).to(bf), "w_up": (H ** -0.5 * _randn(g, E, F, H)).to(bf),
         "offs": offs.cuda(), "most": int(count.max())}
    if case["direction"] == "forward":
        s["x"] = _randn(g, T, H).to(bf)
    else:  # what the forward pass left behind, and the gradient that comes back
        s["gate"], s["up"] = _randn(g, T, F).to(bf), _randn(g, T, F).to(bf)
        s["dh"] = (0.01 * _randn(g, T, F)).to(bf)
    return s


def _prepare_qk(case, g, seed):
    T, A, B, D, dt = case["tokens"], case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    R, P = case["rotary"], 32768
    packed = _randn(g, T, (A + 2 * B) * D).to(dt)  # queries, keys and values of one projection
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    angle = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * freq[None, :]
    # packed sequences: positions run on and start again
    start = _rand(g, T) < 1 / 512
    start[0] = True
    at = torch.arange(T, device="cuda")
    began = torch.cummax(torch.where(start, at, 0), 0).values
    first = (_rand(g, T) * (P - T)).to(torch.int64)[began]
    s = {"q": packed[:, :A * D].view(T, A, D), "k": packed[:, A * D:(A + B) * D].view(T, B, D),
         "w_q": (1 + 0.2 * _randn(g, D)).to(dt), "w_k": (1 + 0.2 * _randn(g, D)).to(dt),
         "cos": torch.cos(angle).float(), "sin": torch.sin(angle).float(),
         "positions": (first + at - began).to(torch.int32), "eps": 1e-6}
    if case["direction"] == "backward":
        s["dq_out"], s["dk_out"] = (0.01 * _randn(g, T, A, D)).to(dt), (0.01 * _randn(g, T, B, D)).to(dt)
    return s


def _prepare_logp(case, g, seed):
    T, V, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    buf = torch.zeros(T, V + case["pad"], dtype=dt, device="cuda")
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 27) // V)
    head = 10 * torch.exp(-torch.arange(32, device="cuda") / 6)  # few tokens are likely
    for a in range(0, T, step):
        b = min(T, a + step)
        z = 2.0 * _randn(g, b - a, V)
        likely = (_rand(g, b - a, 32) * V).to(torch.int64)
        z.scatter_add_(1, likely, (head * (0.3 + _rand(g, b - a, 1))).contiguous())
        rank = (32 * _rand(g, b - a, 1) ** 3).to(torch.int64)
        ids[a:b] = likely.gather(1, rank)[:, 0].to(torch.int32)  # a sampled token is mostly a likely one
        buf[a:b, :V] = z.to(dt)
        del z
    ids[_rand(g, T) < 0.1] = -1  # prompts
    ids[0] = ids[0].clamp(min=0)
    s = {"logits": buf[:, :V], "ids": ids, "tau": case["tau"]}
    if case["direction"] == "backward":
        # what the forward pass left behind, in 32 bits
        top, lns, entropy = _moments(s["logits"], s["tau"])
        live = ids >= 0
        s["stats"] = torch.where(live[:, None], torch.stack([top, lns], 1), 0.0)
        s["entropy"] = torch.where(live, entropy, 0.0)
        s["dlogp"] = _randn(g, T) / T  # advantages
        s["dentropy"] = torch.full((T,), -0.01 / T, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------------ passes

def run(state):
    case = state["case"]
    if own:
        return {"ffn": _own_ffn, "qk": _own_qk, "logp": _own_logp}[case["op"]](state, case)
    return {"ffn": _plain_ffn, "qk": _plain_qk, "logp": _plain_logp}[case["op"]](state, case)


# The package's entry points, with the outputs and workspaces that a training loop keeps from step to step.

def _own_ffn(s, case):
    import deterministic_gradient_reduction_gb300 as dgr
    T, H, F, E = case["tokens"], case["width"], case["hidden"], case["experts"]
    if "ws" not in s:
        s["ws"] = dgr.workspace(dgr.gated_ffn_workspace_bytes(T, H, F, E))
        wide = lambda: torch.empty(T, F, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        if case["direction"] == "forward":
            s["out"] = {"h": wide(), "gate": wide(), "up": wide()} if case["keep"] else {"h": wide()}
        else:
            s["out"] = {"dx": torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), "dgate": wide(), "dup": wide()}
    if case["direction"] == "forward":
        dgr.gated_ffn(s["x"], s["w_gate"], s["w_up"], offs=s["offs"], act=case["act"], ws=s["ws"], **s["out"])
        return s["out"]
    return dgr.gated_ffn_backward(s["dh"], s["gate"], s["up"], s["w_gate"], s["w_up"], offs=s["offs"], act=case["act"],
                                  ws=s["ws"], **s["out"])


def _own_qk(s, case):
    import deterministic_gradient_reduction_gb300 as dgr
    T, A, B, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if "ws" not in s:
        s["ws"] = dgr.workspace(dgr.qk_norm_rope_workspace_bytes(T, A, B, D))
        like = lambda heads: torch.empty(T, heads, D, dtype=s["q"].dtype, device="cuda")  # noqa: E731
        s["out"] = {"q_out": like(A), "k_out": like(B)}
        if case["direction"] == "backward":
            s["out"] = {"dq": like(A), "dk": like(B), "dw_q": torch.empty(D, device="cuda"),
                        "dw_k": torch.empty(D, device="cuda")}
    same = dict(w_q=s["w_q"], w_k=s["w_k"], eps=s["eps"], interleaved=case["interleaved"], ws=s["ws"])
    if case["direction"] == "forward":
        q, k = dgr.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["positions"], **same, **s["out"])
        return {"q": q, "k": k}
    return dgr.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["cos"], s["sin"], s["positions"], **same,
                                     **s["out"])


def _own_logp(s, case):
    import deterministic_gradient_reduction_gb300 as dgr
    z, K = s["logits"], case["top"]
    T, V = z.shape
    if "out" not in s:
        if case["direction"] == "forward":
            f32 = lambda *shape: torch.empty(*shape, device="cuda")  # noqa: E731
            s["ws"] = dgr.workspace(dgr.token_logprobs_workspace_bytes(T))
            s["out"] = {"logp": f32(T), "entropy": f32(T), "lse": f32(T), "stats": f32(T, 2)}
            if K:
                s["out"].update(top_ids=torch.empty(T, K, dtype=torch.int32, device="cuda"), top_logits=f32(T, K),
                                top_logp=f32(T, K))
        else:
            s["out"] = torch.empty(T, V, dtype=z.dtype, device="cuda")
    if case["direction"] == "forward":
        return dgr.token_logprobs(z, s["ids"], tau=s["tau"], top=K, ws=s["ws"], **s["out"])
    return {"dlogits": dgr.token_logprobs_backward(z, s["ids"], s["stats"], s["entropy"], dlogp=s["dlogp"],
                                                   dentropy=s["dentropy"], tau=s["tau"], dlogits=s["out"])}


# The plain forms: torch operations in 32 bits, rounded once at the end.

def _slots(offs, most, T):
    """Rows of every expert side by side: the row in each of its `most` places (T: none), and each row's place."""
    rows = offs[:-1, None] + torch.arange(most, device="cuda")[None, :]
    rows = torch.where(rows < offs[1:, None], rows, T)
    t = torch.arange(T, device="cuda")
    expert = (torch.searchsorted(offs, t, right=True) - 1)
    return rows, expert * most + t - offs[expert]


def _padded(v, rows):
    """v's rows in their places, zeros in the empty ones."""
    v = torch.cat([v, torch.zeros(1, v.shape[1], device="cuda")])
    return v[rows.reshape(-1)].reshape(*rows.shape, v.shape[1])


GELU = math.sqrt(2 / math.pi), 0.044715


def _act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return 0.5 * v * (1 + torch.tanh(GELU[0] * (v + GELU[1] * v * v * v)))


def _act_slope(v, name):
    if name == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    t = torch.tanh(GELU[0] * (v + GELU[1] * v * v * v))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * GELU[0] * (1 + 3 * GELU[1] * v * v)


def _plain_ffn(s, case):
    T, bf = case["tokens"], torch.bfloat16
    rows, place = _slots(s["offs"], s["most"], T)
    w_gate, w_up = s["w_gate"].float(), s["w_up"].float()
    if case["direction"] == "forward":
        x = _padded(s["x"].float(), rows)
        gate = torch.bmm(x, w_gate.transpose(1, 2)).flatten(0, 1)[place]
        up = torch.bmm(x, w_up.transpose(1, 2)).flatten(0, 1)[place]
        out = {"h": (_act(gate, case["act"]) * up).to(bf)}
        if case["keep"]:
            out.update(gate=gate.to(bf), up=up.to(bf))
        return out
    dh, gate, up = s["dh"].float(), s["gate"].float(), s["up"].float()
    dgate, dup = dh * up * _act_slope(gate, case["act"]), dh * _act(gate, case["act"])
    dx = torch.bmm(_padded(dgate, rows), w_gate) + torch.bmm(_padded(dup, rows), w_up)
    return {"dx": dx.flatten(0, 1)[place].to(bf), "dgate": dgate.to(bf), "dup": dup.to(bf)}


def _turn(v, c, s, interleaved):
    """The pairs of v's first elements turned by their angles; what is behind them stays."""
    R = 2 * c.shape[-1]
    a, b = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
    x, y = a * c - b * s, b * c + a * s
    turned = torch.stack([x, y], -1).flatten(-2) if interleaved else torch.cat([x, y], -1)
    return torch.cat([turned, v[..., R:]], -1)


def _plain_qk(s, case):
    at = s["positions"].long()
    c, n, inter, eps, dt = s["cos"][at][:, None], s["sin"][at][:, None], case["interleaved"], s["eps"], s["q"].dtype
    out = {}
    for name in ("q", "k"):
        v, w = s[name].float(), s["w_" + name].float()
        r = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
        if case["direction"] == "forward":
            out[name] = _turn(v * r * w, c, n, inter).to(dt)
            continue
        d = _turn(s["d" + name + "_out"].float(), c, -n, inter)
        hat = v * r
        out["dw_" + name] = (d * hat).sum((0, 1))
        d = d * w
        out["d" + name] = (r * (d - hat * (d * hat).mean(-1, keepdim=True))).to(dt)
    return out


def _moments(logits, tau):
    """Maximum, ln of the sum of exp((z - maximum) / tau), entropy of every row."""
    z = logits.float()
    top = z.amax(1)
    z = (z - top[:, None]) * (1.0 / tau)
    e = torch.exp(z)
    total = e.sum(1)
    lns = torch.log(total)
    return top, lns, lns - (e * z).sum(1) / total


def _plain_logp(s, case):
    logits, ids, k = s["logits"], s["ids"], 1.0 / s["tau"]
    T, V = logits.shape
    live = ids >= 0
    at = ids.clamp(min=0).to(torch.int64)[:, None]
    if case["direction"] == "backward":
        z = (logits.float() - s["stats"][:, :1]) * k - s["stats"][:, 1:]  # ln p
        p = torch.exp(z)
        a, b = s["dlogp"][:, None] * k, s["dentropy"][:, None] * k
        d = -p * (a + b * (z + s["entropy"][:, None]))
        d.scatter_add_(1, at, a)
        return {"dlogits": torch.where(live[:, None], d, 0.0).to(logits.dtype)}
    top, lns, entropy = _moments(logits, s["tau"])
    logp = (logits.gather(1, at)[:, 0].float() - top) * k - lns
    zero = lambda v: torch.where(live, v, 0.0)  # noqa: E731
    out = {"logp": zero(logp), "entropy": zero(entropy), "lse": zero(top * k + lns),
           "stats": torch.where(live[:, None], torch.stack([top, lns], 1), 0.0)}
    if case["top"]:
        # by value, then by the lowest index: both in one whole number
        bits = (logits.float() + 0.0).view(torch.int32).to(torch.int64)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
        best = (order * (1 << 32) - torch.arange(V, device="cuda")).topk(case["top"], dim=1).values
        index = -best % (1 << 32)
        value = logits.gather(1, index).float()
        out["top_ids"] = torch.where(live[:, None], index, -1).to(torch.int32)
        out["top_logits"] = torch.where(live[:, None], value, -math.inf)
        out["top_logp"] = torch.where(live[:, None], (value - top[:, None]) * k - lns[:, None], -math.inf)
    return out


# ------------------------------------------------------------------------------------------------------ work, 64 bits

def work(case):
    if case["op"] == "ffn":
        T, H, F, E = case["tokens"], case["width"], case["hidden"], case["experts"]
        weights = 4 * min(E, T) * F * H  # an expert without rows is not read
        if case["direction"] == "forward":
            return {"bytes": 2 * T * H + weights + 8 * (E + 1) + 2 * T * F * (3 if case["keep"] else 1), "flops": 4 * T * H * F}
        return {"bytes": 2 * T * H + weights + 8 * (E + 1) + 10 * T * F, "flops": 4 * T * H * F}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "qk":
        T, D = case["tokens"], case["dim"]
        n = T * (case["heads"] + case["kv_heads"]) * D
        side = T * (4 + 4 * case["rotary"]) + 2 * D * es
        if case["direction"] == "forward":
            return {"bytes": 2 * n * es + side, "flops": 7 * n}
        return {"bytes": 3 * n * es + side + 8 * D, "flops": 14 * n}
    T, V, K = case["rows"], case["vocab"], case["top"]
    if case["direction"] == "forward":
        return {"bytes": T * V * es + T * (4 + 20 + 12 * K), "flops": 6 * T * V}
    return {"bytes": 2 * T * V * es + T * 24, "flops": 8 * T * V}


def exact(case, seed):
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "qk": _exact_qk, "logp": _exact_logp}[case["op"]](s, case)


def _exact_ffn(s, case):
    """Expert by expert; the gradient by automatic differentiation of the products."""
    offs = s["offs"].tolist()
    act = torch.nn.functional.silu if case["act"] == "silu" else lambda v: torch.nn.functional.gelu(v, approximate="tanh")
    parts = []
    for e in range(case["experts"]):
        rows = slice(offs[e], offs[e + 1])
        if offs[e] == offs[e + 1]:
            continue
        w1, w2 = s["w_gate"][e].double(), s["w_up"][e].double()
        if case["direction"] == "forward":
            x = s["x"][rows].double()
            a, b = x @ w1.t(), x @ w2.t()
            parts.append({"h": act(a) * b, "gate": a, "up": b} if case["keep"] else {"h": act(a) * b})
        else:
            a, b = s["gate"][rows].double().requires_grad_(), s["up"][rows].double().requires_grad_()
            da, db = torch.autograd.grad(act(a) * b, (a, b), s["dh"][rows].double())
            parts.append({"dx": da @ w1 + db @ w2, "dgate": da, "dup": db})
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_qk(s, case):
    """The rotation as a product of complex numbers, the gradient by automatic differentiation."""
    at, R = s["positions"].long(), case["rotary"]
    turn = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
    out = {}
    for name in ("q", "k"):
        v = s[name].double().clone().requires_grad_(case["direction"] == "backward")
        w = s["w_" + name].double().requires_grad_(case["direction"] == "backward")
        n = torch.nn.functional.rms_norm(v, (v.shape[-1],), w, s["eps"])
        pairs = n[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
        pairs = pairs if case["interleaved"] else pairs.transpose(-1, -2)
        got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        got = (got if case["interleaved"] else got.transpose(-1, -2)).flatten(-2)
        got = torch.cat([got, n[..., R:]], -1)
        if case["direction"] == "forward":
            out[name] = got
        else:
            out["d" + name], out["dw_" + name] = torch.autograd.grad(got, (v, w), s["d" + name + "_out"].double())
    return out


def _exact_logp(s, case):
    """In slices of rows, by log_softmax; the gradient of p ln p from its Jacobian."""
    T, V = s["logits"].shape
    tau, live = float(case["tau"]), s["ids"] >= 0
    parts = []
    step = max(1, (1 << 26) // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        z = s["logits"][a:b].double()
        lp = torch.log_softmax(z / tau, dim=1)
        p = torch.exp(lp)
        entropy = torch.special.entr(p).sum(1)
        on = live[a:b].double()
        at = s["ids"][a:b].long().clamp(min=0)[:, None]
        if case["direction"] == "backward":
            g = torch.zeros_like(p).scatter_(1, at, 1.0) - p
            d = g * s["dlogp"][a:b, None].double() - p * (lp + entropy[:, None]) * s["dentropy"][a:b, None].double()
            d = d * (on / tau)[:, None]
            parts.append({"dlogits": d.to(torch.float64 if T * V < 1 << 27 else torch.float32)})
        else:
            top = z.amax(1)
            lse = torch.logsumexp(z / tau, 1)
            got = {"logp": lp.gather(1, at)[:, 0] * on, "entropy": entropy * on, "lse": lse * on,
                   "stats": torch.stack([top, torch.logsumexp((z - top[:, None]) / tau, 1)], 1) * on[:, None]}
            if case["top"]:
                value = z.topk(case["top"], dim=1).values
                none = (on == 0)[:, None]
                got.update(top_logits=value.masked_fill(none, -math.inf),
                           top_logp=(value / tau - lse[:, None]).masked_fill(none, -math.inf))
            parts.append(got)
        del z, lp, p
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["top"]:
        out["top_ids"] = None
    return out
