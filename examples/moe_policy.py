"""Policy-gradient steps of a small mixture-of-experts transformer block, with a teacher's lists for distillation.

The step runs forward and backward through the library's operators, with plain matrix products and a plain softmax
attention between them:

  forward   block_norm, qk_norm_rope (queries and keys of packed sequences), block_norm (behind the attention),
            topk_canonicalize and router_balance (routing), gated_ffn (the experts), block_norm, token_logprobs
  backward  token_logprobs_backward (over the logits' own memory), block_norm_backward, ordered_rowdot_dprob,
            gated_ffn_backward with grouped_wgrad_accumulate for its weights, det_index_add, router_balance_backward,
            qk_norm_rope_backward, block_norm_backward

The loss is -sum_t advantage_t ln p(token_t) - BONUS sum_t entropy_t over the tokens that carry one (prompts do not),
over their number, and the routers' balance loss. Every reduction of the library has a fixed order: two runs from the
same seed end in the same bits, as far as the plain products between do.

    python examples/moe_policy.py [steps]
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import deterministic_gradient_reduction_gb300 as dgr  # noqa: E402

H, HEADS, KV, D, EXPERTS, TOPK, F, VOCAB = 256, 4, 2, 64, 4, 2, 128, 1000
COEFF, BONUS, EPS, TAU, LIST = 0.01, 0.01, 1e-6, 1.0, 16


def tables(positions: int, device="cuda"):
    """Cosines and sines of every position's angles."""
    freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device=device) / D)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def parameters(seed: int, device="cuda") -> dict:
    """Master weights in fp32."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s, scale: scale * torch.randn(*s, generator=g, device=device)  # noqa: E731
    one = lambda n: torch.ones(n, device=device)  # noqa: E731
    return {"embed": r(VOCAB, H, scale=0.5), "norm1": one(H), "qkv": r(H, (HEADS + 2 * KV) * D, scale=H ** -0.5),
            "q_norm": one(D), "k_norm": one(D), "proj": r(HEADS * D, H, scale=H ** -0.5), "norm2": one(H),
            "router": r(H, EXPERTS, scale=H ** -0.5), "w_gate": r(EXPERTS, F, H, scale=H ** -0.5),
            "w_up": r(EXPERTS, F, H, scale=H ** -0.5), "w_down": r(EXPERTS, H, F, scale=F ** -0.5), "norm3": one(H),
            "out": r(H, VOCAB, scale=H ** -0.5)}


def batch(sequences: int, length: int, seed: int, device="cuda") -> dict:
    """Packed sequences of tokens, the sampled ones that follow, their advantages; the first quarter is the prompt."""
    g = torch.Generator(device=device).manual_seed(seed)
    T = sequences * length
    ids = torch.randint(0, VOCAB, (T,), generator=g, device=device, dtype=torch.int32)
    positions = torch.arange(length, device=device, dtype=torch.int32).repeat(sequences)
    ids[positions < length // 4] = -1
    return {"x": torch.randint(0, VOCAB, (T,), generator=g, device=device), "ids": ids, "positions": positions,
            "advantage": torch.randn(T, generator=g, device=device), "length": length}


def attend(q, k, v, length):
    """Causal attention within each sequence, in fp32; (output, probabilities)."""
    S = q.shape[0] // length
    split = lambda t: t.view(S, length, t.shape[1], D).transpose(1, 2)  # noqa: E731
    q, k, v = split(q), split(k).repeat_interleave(HEADS // KV, 1), split(v).repeat_interleave(HEADS // KV, 1)
    score = (q @ k.transpose(2, 3)) * D ** -0.5
    score = score.masked_fill(torch.ones(length, length, dtype=torch.bool, device=q.device).triu(1), -float("inf"))
    p = torch.softmax(score, -1)
    return (p @ v).transpose(1, 2).reshape(S * length, HEADS * D), p


def attend_backward(do, p, q, k, v, length):
    """Gradients to q, k and v; those of a shared key's or value's heads added in their order."""
    S = q.shape[0] // length
    split = lambda t: t.view(S, length, t.shape[1], D).transpose(1, 2)  # noqa: E731
    back = lambda t: t.transpose(1, 2).reshape(S * length, -1, D)  # noqa: E731
    q, do = split(q), split(do.view(S * length, HEADS, D))
    k, v = split(k).repeat_interleave(HEADS // KV, 1), split(v).repeat_interleave(HEADS // KV, 1)
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * D ** -0.5
    shared = lambda t: t.view(S, KV, HEADS // KV, length, D).sum(2)  # noqa: E731
    return back(ds @ k), back(shared(ds.transpose(2, 3) @ q)), back(shared(p.transpose(2, 3) @ do))


def step(P: dict, data: dict):
    """(policy loss, balance loss, gradients in fp32) of one batch."""
    T, length = data["x"].numel(), data["length"]
    bf, b16 = {k: v.to(torch.bfloat16) for k, v in P.items()}, torch.bfloat16
    cos, sin = tables(length, data["x"].device)
    norms = dict(w_q=bf["q_norm"], w_k=bf["k_norm"], eps=EPS)
    # ---- forward: attention ----
    x = bf["embed"][data["x"]]
    _, u1 = dgr.block_norm(x, w_pre=bf["norm1"], eps=EPS)
    packed = (u1.float() @ bf["qkv"].float()).to(b16)
    q = packed[:, :HEADS * D].view(T, HEADS, D)
    k = packed[:, HEADS * D:(HEADS + KV) * D].view(T, KV, D)
    v = packed[:, (HEADS + KV) * D:].view(T, KV, D).float()
    qr, kr = dgr.qk_norm_rope(q, k, cos, sin, data["positions"], **norms)
    mixed, p_att = attend(qr.float(), kr.float(), v, length)
    mixed = mixed.to(b16)
    y1 = (mixed.float() @ bf["proj"].float()).to(b16)
    h1, u2 = dgr.block_norm(x, y1, w_pre=bf["norm2"], eps=EPS)
    # ---- forward: experts ----
    scores = u2.float() @ bf["router"].float()
    top = scores.topk(TOPK, dim=1)
    chosen, _, prob = dgr.topk_canonicalize(top.indices.to(torch.int32), top.values)
    balance, counts, tokens = dgr.router_balance(scores, chosen, COEFF)
    order = torch.argsort(chosen.reshape(-1), stable=True)  # rows (token, slot) grouped by expert
    token = order // TOPK
    offs = torch.cat([torch.zeros(1, dtype=torch.int64, device=x.device), counts[0].long().cumsum(0)])
    cuts = offs.tolist()
    rows = [slice(cuts[e], cuts[e + 1]) for e in range(EXPERTS)]
    xe = u2[token]
    gate, up = (torch.empty(T * TOPK, F, dtype=b16, device=x.device) for _ in range(2))
    he = dgr.gated_ffn(xe, bf["w_gate"], bf["w_up"], offs=offs, gate=gate, up=up)
    ye = torch.cat([he[r].float() @ bf["w_down"][e].float().t() for e, r in enumerate(rows)]).to(b16)
    back = torch.argsort(order)
    y2 = (ye[back].reshape(T, TOPK, H).float() * prob[:, :, None]).sum(1).to(b16)
    h2, u3 = dgr.block_norm(h1, y2, w_pre=bf["norm3"], eps=EPS)
    # ---- the policy's loss ----
    logits = (u3.float() @ bf["out"].float()).to(b16)
    got = dgr.token_logprobs(logits, data["ids"], tau=TAU)
    n = (data["ids"] >= 0).sum()
    loss = -((data["advantage"] * got["logp"]).sum() + BONUS * got["entropy"].sum()) / n
    dz = dgr.token_logprobs_backward(logits, data["ids"], got["stats"], got["entropy"], dlogp=-data["advantage"] / n,
                                     dentropy=(-BONUS / n).expand(T).contiguous(), tau=TAU, dlogits=logits).float()
    # ---- backward: experts ----
    g = {"out": u3.float().t() @ dz}
    b = dgr.block_norm_backward(h2, y2, None, (dz @ bf["out"].float().t()).to(b16), w_pre=bf["norm3"], eps=EPS)
    g["norm3"] = b["dw_pre"]
    dy_rows = b["dy"][token]
    dprob = torch.zeros(T * TOPK, device=x.device)
    dgr.ordered_rowdot_dprob(dy_rows, ye, dprob)
    dprob = dprob[back].reshape(T, TOPK)
    dye = (dy_rows.float() * prob.reshape(-1)[order][:, None]).to(b16)
    g["w_down"] = torch.stack([dye[r].float().t() @ he[r].float() for r in rows])
    dhe = torch.cat([dye[r].float() @ bf["w_down"][e].float() for e, r in enumerate(rows)]).to(b16)
    g["w_gate"], g["w_up"] = (torch.zeros(EXPERTS, F, H, device=x.device) for _ in range(2))
    f = dgr.gated_ffn_backward(dhe, gate, up, bf["w_gate"], bf["w_up"], offs=offs, dgate=gate, dup=up, x=xe,
                               dw_gate=g["w_gate"], dw_up=g["w_up"])  # the products' gradients in their place
    du2 = torch.zeros(T + 1, H, device=x.device)
    dgr.det_index_add(du2, f["dx"].float(), token.to(torch.int32))
    dchosen = prob * (dprob - (prob * dprob).sum(1, keepdim=True))
    dscores = torch.zeros_like(scores).scatter_(1, chosen.long(), dchosen)
    dgr.router_balance_backward(scores, counts, tokens, TOPK, COEFF, dlogits=dscores, accumulate=True)
    g["router"] = u2.float().t() @ dscores
    du2 = (du2[:T] + dscores @ bf["router"].float().t()).to(b16)
    # ---- backward: attention ----
    b = dgr.block_norm_backward(h1, y1, b["dx"], du2, w_pre=bf["norm2"], eps=EPS)
    g["norm2"] = b["dw_pre"]
    g["proj"] = mixed.float().t() @ b["dy"].float()
    dq, dk, dv = attend_backward(b["dy"].float() @ bf["proj"].float().t(), p_att, qr.float(), kr.float(), v, length)
    dpacked = torch.empty_like(packed)
    dpacked[:, (HEADS + KV) * D:] = dv.reshape(T, -1).to(b16)
    a = dgr.qk_norm_rope_backward(dq.to(b16), dk.to(b16), q, k, cos, sin, data["positions"], **norms,
                                  dq=dpacked[:, :HEADS * D].view(T, HEADS, D),
                                  dk=dpacked[:, HEADS * D:(HEADS + KV) * D].view(T, KV, D))
    g["q_norm"], g["k_norm"] = a["dw_q"], a["dw_k"]
    g["qkv"] = u1.float().t() @ dpacked.float()
    n1 = dgr.block_norm_backward(x, None, b["dx"], (dpacked.float() @ bf["qkv"].float().t()).to(b16), w_pre=bf["norm1"], eps=EPS)
    g["norm1"] = n1["dw_pre"]
    g["embed"] = torch.zeros(VOCAB + 1, H, device=x.device)
    dgr.det_index_add(g["embed"], n1["dx"].float(), data["x"].to(torch.int32))
    g["embed"] = g["embed"][:VOCAB]
    return loss, balance, g


def teacher_lists(logits: torch.Tensor, tau: float = TAU):
    """What topk_distill takes of a teacher: the ids and logits of its top alternatives, and its logsumexp."""
    t = dgr.token_logprobs(logits, tau=tau, top=LIST)
    return t["top_ids"], t["top_logits"], t["lse"]


def train(steps: int, sequences: int = 8, length: int = 64, seed: int = 0, rate: float = 1.0):
    """Plain gradient descent; (losses, the weights at the end)."""
    P, losses = parameters(seed), []
    for i in range(steps):
        loss, balance, g = step(P, batch(sequences, length, 100 + i))
        losses.append((loss, balance))
        for k in P:
            P[k] -= rate * g[k]
    return [(float(a), float(b)) for a, b in losses], P


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 10
    losses, _ = train(steps)
    for i, (loss, balance) in enumerate(losses):
        print(f"step {i:3d}  policy {loss:.5f}  balance {balance:.5f}")


if __name__ == "__main__":
    main()
