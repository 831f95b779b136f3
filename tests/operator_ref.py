"""Plain 64-bit forms of the router balance loss, the block norms and the distillation loss.

Written from the formulas with torch's elementary operations on CPU tensors. The losses are
differentiable, so their gradients come from torch's autograd and not from the formulas that the
kernels use; test_operator_ref.py holds them against finite differences.

Each *_bound function gives the error that binary32 arithmetic may leave: u = 2^-24 times the number
of roundings on the path times the sum of the magnitudes that meet there, plus half a unit of the
output's own type (`ulp`).
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def half_ulp(dtype) -> float:
    """Largest relative error of one rounding to nearest: 2^-p for p bits of significand (bf16: 8)."""
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def d(t):
    return None if t is None else t.detach().cpu().double()


# ------------------------------------------------------------------------------------------------ router balance

def balance_scores(x, score):
    if score == "sigmoid":
        x = torch.nn.functional.logsigmoid(x)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top))
    s = e.sum(1, keepdim=True)
    return e / torch.where(s == 0, torch.ones_like(s), s)


def balance(logits, ids, coeff, offs=None, mask=None, score="softmax"):
    """(loss, counts [G, E], tokens [G]); logits may require a gradient."""
    N, E = logits.shape
    K = ids.shape[1]
    cuts = [0, N] if offs is None else [int(v) for v in offs]
    G = len(cuts) - 1
    counts = torch.zeros(G, E, dtype=torch.int64)
    tokens = torch.zeros(G, dtype=torch.int64)
    loss = logits.new_zeros(())
    for g in range(G):
        rows = [t for t in range(cuts[g], cuts[g + 1]) if mask is None or mask[t]]
        tokens[g] = len(rows)
        if not rows:
            continue
        for i in ids[rows].reshape(-1).tolist():
            if 0 <= i < E:
                counts[g, i] += 1
        p = balance_scores(logits[rows], score)
        loss = loss + coeff * E / (G * K * len(rows) ** 2) * (counts[g].double() * p.sum(0)).sum()
    return loss, counts, tokens


def finite_range(x):
    """Largest distance of a finite logit from its row's maximum (in powers of two)."""
    f = torch.where(torch.isfinite(x), x, torch.full_like(x, math.nan))
    lo = torch.nan_to_num(f, nan=math.inf).amin(1)
    hi = torch.nan_to_num(f, nan=-math.inf).amax(1)
    r = (hi - lo)[torch.isfinite(hi - lo)]
    return 1.4427 * float(r.max()) if r.numel() else 0.0


# ---------------------------------------------------------------------------------------------------- block norm

def rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def block_norm(x, y, w_post, gate, res_scale, w_pre, eps):
    g = 1.0 if gate is None else gate
    if y is None:
        h = x
    else:
        n = y if w_post is None else y * rms(y, eps) * w_post
        h = res_scale * x + g * n
    return h, None if w_pre is None else h * rms(h, eps) * w_pre


def block_norm_bounds(x, y, w_post, gate, res_scale, w_pre, eps, dtype):
    """Bounds of the errors of h and u. A norm's factor comes from a sum of at most 16 + 5 + 32 steps
    and a root: with the products around it, 64 roundings at most."""
    h, u = block_norm(x, y, w_post, gate, res_scale, w_pre, eps)
    dh = torch.zeros_like(h)
    if y is not None:
        n = h - res_scale * x
        dh = 64 * U * ((res_scale * x).abs() + n.abs())
    bh = dh + half_ulp(dtype) * h.abs()
    bu = None
    if u is not None:
        size = torch.sqrt((h * h).sum(1, keepdim=True)).clamp(min=1e-300)
        rel = 64 * U + torch.sqrt((dh * dh).sum(1, keepdim=True)) / size
        bu = w_pre.abs() * rms(h, eps) * (dh + h.abs() * rel) + half_ulp(dtype) * u.abs()
    return bh, bu


def block_norm_grads(h, y, dh, du, w_post, gate, res_scale, w_pre, eps):
    """Gradients by autograd, with h as an input of its own: x = (h - gate n) / res_scale is not
    needed, as u depends on x and y through h alone."""
    T, H = (du if du is not None else dh).shape
    out = {}
    if w_pre is not None:
        hv, wv = h.clone().requires_grad_(), w_pre.clone().requires_grad_()
        gh, gw = torch.autograd.grad(hv * rms(hv, eps) * wv, (hv, wv), du)
        out["dw_pre"] = gw
        D = gh if dh is None else dh + gh
    else:
        D = dh
    out["D"] = D
    out["dx"] = res_scale * D
    if y is not None:
        leaves = {"dy": y.clone().requires_grad_()}
        if w_post is not None:
            leaves["dw_post"] = w_post.clone().requires_grad_()
        if gate is not None:
            leaves["dgate"] = gate.clone().requires_grad_()
        n = leaves["dy"] if w_post is None else leaves["dy"] * rms(leaves["dy"], eps) * leaves["dw_post"]
        v = n if gate is None else n * leaves["dgate"]
        out.update(zip(leaves, torch.autograd.grad(v, list(leaves.values()), D)))
    return out


def block_norm_grad_bounds(h, y, dh, du, w_post, gate, res_scale, w_pre, eps):
    """Bounds before the outputs' own rounding: magnitudes of the terms of each gradient, times 128
    roundings in a row's own arithmetic; the sums over tokens add one rounding for each row of a slot
    and each slot of a way, at most T."""
    T, H = (du if du is not None else dh).shape
    one = torch.ones(1, dtype=torch.float64)
    size = torch.zeros(T, H, dtype=torch.float64) if dh is None else dh.abs()
    b = {}
    rows = min(T, 64 + T // 256)
    if w_pre is not None:
        r2 = rms(h, eps)
        v = (du * w_pre).abs()
        size = size + r2 * v + h.abs() * r2 ** 3 / H * (v * h.abs()).sum(1, keepdim=True)
        b["dw_pre"] = (128 + rows) * U * (du * h * r2).abs().sum(0)
    b["dx"] = 128 * U * abs(res_scale) * size
    if y is not None:
        g = one if gate is None else gate.abs()
        w = one if w_post is None else w_post.abs()
        r1 = rms(y, eps) if w_post is not None else one
        b["dy"] = 128 * U * r1 * g * w * size
        if w_post is not None:
            b["dy"] = b["dy"] + 128 * U * y.abs() * r1 ** 3 / H * (g * w * size * y.abs()).sum(1, keepdim=True)
            b["dw_post"] = (128 + rows) * U * (g * size * y.abs() * r1).sum(0)
        if gate is not None:
            terms = size * y.abs() * r1 * w
            b["dgate"] = 128 * U * terms.sum(1, keepdim=True) if gate.dim() == 2 else (128 + rows) * U * terms.sum(0)
    return b


# -------------------------------------------------------------------------------------------------------- distill

def distill_rows(z, ids, teacher, tau, teacher_lse=None, weights=None):
    """Row losses; z may require a gradient. Rows of weight 0 or without an entry give 0."""
    T, V = z.shape
    K = ids.shape[1]
    rows = []
    for t in range(T):
        entries = [k for k in range(K) if 0 <= int(ids[t, k]) < V]
        if teacher_lse is None:
            entries = [k for k in entries if float(teacher[t, k]) > -math.inf]
        if not entries or (weights is not None and float(weights[t]) == 0.0):
            rows.append(torch.zeros((), dtype=torch.float64))
            continue
        at = ids[t, entries].long()
        tl = teacher[t, entries] / tau
        log_q = tl - (torch.logsumexp(tl, 0) if teacher_lse is None else teacher_lse[t])
        q = torch.exp(log_q)
        log_p = torch.log_softmax(z[t] / tau, 0)
        keep = q > 0
        L = (q[keep] * (log_q[keep] - log_p[at[keep]])).sum()
        if teacher_lse is not None:
            outside = torch.ones(V, dtype=torch.bool)
            outside[at] = False
            outside &= z[t].detach() > -math.inf
            left = max(0.0, 1.0 - float(q.sum()))
            if left > 0 and bool(outside.any()):
                L = L + left * (math.log(left) - torch.logsumexp(log_p[outside], 0))
        rows.append(L)
    return torch.stack(rows) if rows else torch.zeros(0, dtype=torch.float64)


def distill(z, ids, teacher, tau=1.0, teacher_lse=None, weights=None, scale=1.0):
    """(loss, row losses, gradient of the loss to z)."""
    z = z.clone().requires_grad_()
    rows = distill_rows(z, ids, teacher, tau, teacher_lse, weights)
    w = torch.ones(len(rows), dtype=torch.float64) if weights is None else weights
    loss = scale * (torch.where(w != 0, w, torch.zeros_like(w)) * rows).sum()
    grad = torch.zeros_like(z)
    if loss.requires_grad:
        grad = torch.autograd.grad(loss, z)[0]
        grad = torch.where(z == -math.inf, torch.zeros_like(grad), grad)  # autograd has 0 * inf there
    return loss.detach(), rows.detach(), grad


def distill_bounds(z, ids, teacher, tau, teacher_lse, weights, scale, dtype, grad):
    """Bounds for (row losses, gradient). R: the largest exponent met (a power of two): its product
    with log2(e) / tau is rounded, so an exponential carries R u; an exponential itself and the sums
    around it stay within 64 u. ln q and ln p carry R u and 64 u of their own size."""
    T, V = z.shape
    fin = torch.where(torch.isfinite(z), z, torch.zeros_like(z)) / tau
    tf = torch.where(torch.isfinite(teacher), teacher, torch.zeros_like(teacher)) / tau
    R = 1.4427 * max(float((2 * fin.abs()).max()), float((2 * tf.abs()).max()),
                     0.0 if teacher_lse is None else float(teacher_lse.abs().max())) + 32
    row = torch.full((T,), (64 + 8 * R) * U, dtype=torch.float64)
    w = torch.ones(T, dtype=torch.float64) if weights is None else weights.abs()
    f = (abs(scale) / tau * w)[:, None]
    # p and q of the entry, each with a relative error; q_r's is absolute, and p_j / p_r <= 1 outside
    p = torch.softmax(torch.where(torch.isnan(z), torch.zeros_like(z), z) / tau, 1)
    g = f * (64 + 4 * R) * U * (p + grad.abs() / f.clamp(min=1e-300))
    if teacher_lse is not None:
        pr = p.clone()
        for t in range(T):
            for k in ids[t].tolist():
                if 0 <= k < V:
                    pr[t, k] = 0
        share = pr / pr.sum(1, keepdim=True).clamp(min=1e-300)
        g = g + f * (64 + 4 * R) * U * share
    return row, g + half_ulp(dtype) * grad.abs()
