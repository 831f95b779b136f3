"""Training steps of a small mixture-of-experts student that is distilled from a teacher's top logits.

One block: norm, router, experts, norm after the experts with a learned gate and a scaled residual, output layer.
The step runs forward and backward through the library's operators, with plain matrix products between them:

  forward   block_norm (before the block), topk_canonicalize (routing weights), router_balance (balance loss, counts),
            block_norm (after the experts, with gate, residual and the output layer's norm), topk_distill
  backward  topk_distill (the loss's gradient, over the logits' own memory), block_norm_backward, ordered_rowdot_dprob
            (routing weights), grouped_wgrad_accumulate and grouped_dbias (experts), det_index_add (tokens' gradients
            gathered from their experts), router_balance_backward

Every reduction in it has a fixed order: two runs from the same seed end in the same bits.

    python examples/moe_distillation.py [steps]
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import deterministic_gradient_reduction_gb300 as dgr  # noqa: E402

H, EXPERTS, TOPK, VOCAB, LIST = 256, 8, 2, 1000, 16
RES_SCALE, COEFF, TAU, EPS = 0.9, 0.01, 2.0, 1e-6


def parameters(seed: int, device="cuda") -> dict:
    """Master weights in fp32."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s, scale: scale * torch.randn(*s, generator=g, device=device)  # noqa: E731
    return {"embed": r(VOCAB, H, scale=0.5), "norm": torch.ones(H, device=device), "router": r(H, EXPERTS, scale=H ** -0.5),
            "experts": r(EXPERTS, H, H, scale=H ** -0.5), "bias": torch.zeros(EXPERTS, H, device=device),
            "post": torch.ones(H, device=device), "gate": torch.full((H,), 0.5, device=device),
            "pre": torch.ones(H, device=device), "out": r(H, VOCAB, scale=H ** -0.5)}


def batch(tokens: int, seed: int, device="cuda") -> dict:
    """Tokens and the teacher's lists: its top logits, its logsumexp, and weights that leave prompts out."""
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randint(0, VOCAB, (tokens,), generator=g, device=device)
    table = torch.randn(VOCAB, VOCAB, generator=torch.Generator(device=device).manual_seed(7), device=device) * 2.0
    full = table[x]
    top = full.topk(LIST, dim=1)
    return {"x": x, "ids": top.indices.to(torch.int32), "teacher": top.values.contiguous(),
            "lse": torch.logsumexp(full / TAU, dim=1), "weights": (torch.rand(tokens, generator=g, device=device) > 0.1).float()}


def step(P: dict, data: dict):
    """(loss, balance loss, gradients) of one batch; gradients in fp32."""
    T = data["x"].numel()
    bf = {k: v.to(torch.bfloat16) for k, v in P.items()}
    # ---- forward ----
    x = bf["embed"][data["x"]]
    _, u0 = dgr.block_norm(x, w_pre=bf["norm"], eps=EPS)
    scores = u0.float() @ bf["router"].float()
    top = scores.topk(TOPK, dim=1)
    ids, _, prob = dgr.topk_canonicalize(top.indices.to(torch.int32), top.values)
    balance, counts, tokens = dgr.router_balance(scores, ids, COEFF)
    # rows (token, slot) grouped by expert, in the tokens' order within each
    order = torch.argsort(ids.reshape(-1), stable=True)
    token = order // TOPK
    offs = torch.cat([torch.zeros(1, dtype=torch.int64, device=x.device), counts[0].long().cumsum(0)])
    xe = u0[token]
    expert = ids.reshape(-1)[order].long()
    ye = torch.empty_like(xe)
    cuts = offs.tolist()
    for e in range(EXPERTS):
        ye[cuts[e]:cuts[e + 1]] = (xe[cuts[e]:cuts[e + 1]].float() @ bf["experts"][e].float().t() + bf["bias"][e].float()).to(torch.bfloat16)
    back = torch.argsort(order)  # where each (token, slot) went
    y = (ye[back].reshape(T, TOPK, H).float() * prob[:, :, None]).sum(1).to(torch.bfloat16)
    h, u = dgr.block_norm(x, y, w_post=bf["post"], gate=bf["gate"], res_scale=RES_SCALE, w_pre=bf["pre"], eps=EPS)
    logits = (u.float() @ bf["out"].float()).to(torch.bfloat16)
    lists, teacher, _ = dgr.topk_canonicalize(data["ids"], data["teacher"])
    loss, _ = dgr.topk_distill(logits, lists, teacher, tau=TAU, teacher_lse=data["lse"], weights=data["weights"],
                               scale=TAU * TAU / T, dlogits=logits)  # the gradient takes the logits' place
    # ---- backward ----
    g = {}
    dz = logits.float()
    g["out"] = u.float().t() @ dz
    du = (dz @ bf["out"].float().t()).to(torch.bfloat16)
    b = dgr.block_norm_backward(h, y, None, du, w_post=bf["post"], gate=bf["gate"], res_scale=RES_SCALE, w_pre=bf["pre"], eps=EPS)
    g["post"], g["gate"], g["pre"] = b["dw_post"], b["dgate"], b["dw_pre"]
    dy_rows = b["dy"][token]
    dprob = torch.zeros(T * TOPK, device=x.device)
    dgr.ordered_rowdot_dprob(dy_rows, ye, dprob)
    dprob = dprob[back].reshape(T, TOPK)
    dye = (dy_rows.float() * prob.reshape(-1)[order][:, None]).to(torch.bfloat16)
    g["experts"] = torch.zeros(EXPERTS, H, H, device=x.device)
    dgr.grouped_wgrad_accumulate(dye, xe, offs, g["experts"])
    g["bias"] = torch.zeros(EXPERTS, H, device=x.device)
    dgr.grouped_dbias(dye, offs, g["bias"])
    dxe = torch.empty(T * TOPK, H, device=x.device)
    for e in range(EXPERTS):
        dxe[cuts[e]:cuts[e + 1]] = dye[cuts[e]:cuts[e + 1]].float() @ bf["experts"][e].float()
    du0 = torch.zeros(T + 1, H, device=x.device)
    dgr.det_index_add(du0, dxe, token.to(torch.int32))
    # the router: its softmax over the chosen experts, and the balance loss
    dchosen = prob * (dprob - (prob * dprob).sum(1, keepdim=True))
    dscores = torch.zeros_like(scores).scatter_(1, ids.long(), dchosen)
    dgr.router_balance_backward(scores, counts, tokens, TOPK, COEFF, dlogits=dscores, accumulate=True)
    g["router"] = u0.float().t() @ dscores
    du0 = du0[:T] + dscores @ bf["router"].float().t()
    n = dgr.block_norm_backward(x, None, b["dx"], du0.to(torch.bfloat16), w_pre=bf["norm"], eps=EPS)
    g["norm"] = n["dw_pre"]
    g["embed"] = torch.zeros(VOCAB + 1, H, device=x.device)
    dgr.det_index_add(g["embed"], n["dx"].float(), data["x"].to(torch.int32))
    g["embed"] = g["embed"][:VOCAB]
    return loss, balance, g


def train(steps: int, tokens: int = 2048, seed: int = 0, rate: float = 20.0):
    """Plain gradient descent; (losses, the weights at the end)."""
    P, losses = parameters(seed), []
    for i in range(steps):
        loss, balance, g = step(P, batch(tokens, 100 + i))
        losses.append((loss, balance))
        for k in P:
            P[k] -= rate * g[k]
    return [(float(a), float(b)) for a, b in losses], P


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 20
    losses, P = train(steps)
    for i, (loss, balance) in enumerate(losses):
        print(f"step {i:3d}  distillation {loss:.5f}  balance {balance:.5f}")
    again, Q = train(steps)
    same = all(torch.equal(P[k], Q[k]) for k in P) and again == losses
    print("a second run from the same seed ends in", "the same bits" if same else "OTHER bits")


if __name__ == "__main__":
    main()
