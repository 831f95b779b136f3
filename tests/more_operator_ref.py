"""Plain 64-bit forms of the gated feed-forward, the norm and rotation of queries and keys, and the token
log probabilities.

Written from the formulas with torch's elementary operations on CPU tensors, differentiable, so that
gradients come from torch's autograd; test_more_operator_ref.py holds them against finite differences.

The *_bound functions give the error that the arithmetic may leave: U = 2^-24 times the number of
roundings on the path times the sum of the magnitudes that meet there, plus half a unit of the output's
own type.
"""
from __future__ import annotations

import math

import torch

from operator_ref import U, d, half_ulp  # noqa: F401

TINY = 1e-36  # below the range of a normal binary32 product


# ---------------------------------------------------------------------------------------------- gated feed-forward

def inner(v, act):
    return v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)


def activation(v, act):
    return v * torch.sigmoid(inner(v, act))


def ffn(x, w_gate, w_up, offs, act):
    """(h, a, b) of rows grouped by expert; weights [E, F, H]."""
    a, b = [], []
    for e in range(w_gate.shape[0]):
        rows = x[offs[e]:offs[e + 1]]
        a.append(rows @ w_gate[e].t())
        b.append(rows @ w_up[e].t())
    a, b = torch.cat(a), torch.cat(b)
    return activation(a, act) * b, a, b


def product_bound(x, w, offs, by_out=True):
    """A product of K terms on the tensor cores, 16 at a time: each of the 17 aligned terms of a step and its
    sum lose less than a unit of 2^-24 of the largest (19 in all), so 19 / 16 K units of the terms' magnitudes."""
    K = x.shape[1]
    parts = [x[offs[e]:offs[e + 1]].abs() @ (w[e].abs().t() if by_out else w[e].abs()) for e in range(w.shape[0])]
    return (1.2 * K + 20) * U * torch.cat(parts)


def ffn_bounds(x, w_gate, w_up, offs, act):
    h, a, b = ffn(x, w_gate, w_up, offs, act)
    ea, eb = product_bound(x, w_gate, offs), product_bound(x, w_up, offs)
    half = half_ulp(torch.bfloat16)
    # a sigmoid of an exponent s: 4 |s| + 32 roundings at most; |act'| is below 1.2
    s = inner(a, act).abs().clamp(max=200)
    fa = activation(a, act).abs()
    eh = b.abs() * (1.2 * ea + (32 + 4 * s) * U * fa) + (fa + 1.2 * ea) * eb
    return eh + half * (h.abs() + eh) + TINY, ea + half * (a.abs() + ea) + TINY, eb + half * (b.abs() + eb) + TINY


def pre_grads(dh, a, b, act):
    """(da, db) by automatic differentiation."""
    a, b = a.clone().requires_grad_(), b.clone().requires_grad_()
    return torch.autograd.grad(activation(a, act) * b, (a, b), dh)


def pre_grad_bounds(dh, a, b, act):
    da, db = pre_grads(dh, a, b, act)
    v = a.clone().requires_grad_()
    slope = torch.autograd.grad(inner(v, act).sum(), v)[0].abs()
    s = inner(a, act).abs().clamp(max=200)
    g = torch.sigmoid(inner(a, act))
    half = half_ulp(torch.bfloat16)
    turn = a.abs() * slope * g
    # 1 - g loses its relative precision near 0: an absolute unit there
    ea = (dh * b).abs() * U * ((32 + 8 * s) * (g + turn * (1 - g)) + 4 * turn)
    eb = (dh * a).abs() * g * (32 + 4 * s) * U
    return ea + half * (da.abs() + ea) + TINY, eb + half * (db.abs() + eb) + TINY


def dx(dgate, dup, w_gate, w_up, offs):
    return torch.cat([dgate[offs[e]:offs[e + 1]] @ w_gate[e] + dup[offs[e]:offs[e + 1]] @ w_up[e] for e in range(w_gate.shape[0])])


def dx_bound(dgate, dup, w_gate, w_up, offs):
    both = torch.cat([dgate, dup], 1), torch.cat([w_gate, w_up], 1)
    e = product_bound(both[0], both[1], offs, by_out=False)
    return e + half_ulp(torch.bfloat16) * (dx(dgate, dup, w_gate, w_up, offs).abs() + e) + TINY


# -------------------------------------------------------------------------------------------- queries and keys

def turn(n, c, s, interleaved):
    """n [T, heads, D], c and s [T, R/2]."""
    R = 2 * c.shape[1]
    c, s = c[:, None], s[:, None]
    i = torch.arange(R // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y = n.clone()
    y[..., lo] = n[..., lo] * c - n[..., hi] * s
    y[..., hi] = n[..., hi] * c + n[..., lo] * s
    return y


def qk(v, w, c, s, eps, interleaved):
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    return turn(v * r * (1.0 if w is None else w), c, s, interleaved)


def qk_bound(v, w, c, s, eps, interleaved, dtype):
    """A head's factor comes from at most 16 + 5 steps and a root; with the products around it 48 roundings."""
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    n = (v * r * (1.0 if w is None else w)).abs()
    # the two terms of a turned element, A = n c and B = n' s: |A + B| + |A - B| = 2 max(A, B) >= A + B (without the first
    # absolute value the lower half had (A - B) + (A + B) = 2 A alone, which is no bound where B is the larger)
    size = turn(n, c.abs(), -s.abs(), interleaved).abs() + turn(n, c.abs(), s.abs(), interleaved).abs() + 2 * n
    return 48 * U * size + half_ulp(dtype) * qk(v, w, c, s, eps, interleaved).abs() + TINY


def qk_grads(dy, v, w, c, s, eps, interleaved):
    """(dv, dw)."""
    v = v.clone().requires_grad_()
    w = (torch.ones(v.shape[-1], dtype=torch.float64) if w is None else w.clone()).requires_grad_()
    return torch.autograd.grad(qk(v, w, c, s, eps, interleaved), (v, w), dy)


def qk_grad_bounds(dy, v, w, c, s, eps, interleaved, dtype):
    T, heads, D = v.shape
    w = torch.ones(D, dtype=torch.float64) if w is None else w
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    g = turn(dy.abs(), c.abs(), s.abs(), interleaved).abs() + turn(dy.abs(), c.abs(), -s.abs(), interleaved).abs()
    size = r * g * w.abs() + v.abs() * r ** 3 / D * (g * w.abs() * v.abs()).sum(-1, keepdim=True)
    dv, _ = qk_grads(dy, v, w, c, s, eps, interleaved)
    # a lane's heads of a slot, then at most 5 + 8 + 10 + 5 steps
    chain = T * heads // 2432 + heads + 64
    return 64 * U * size + half_ulp(dtype) * dv.abs() + TINY, (64 + chain) * U * (g * v.abs() * r).sum((0, 1)) + TINY


# -------------------------------------------------------------------------------------------- log probabilities

def logp_rows(z, tau):
    """(ln p, entropy, lse) with masked places (-inf) as 0 in the sums; a row of nothing else: -inf, 0, -inf."""
    none = (z == -math.inf).all(1, keepdim=True)
    x = torch.where(none, torch.zeros_like(z), z) / tau
    m = x.detach().amax(1, keepdim=True)
    # the maximum first: beside one of 1e38 even 64 bits lose the logarithm of the sum
    lns = torch.log(torch.exp(x - m).sum(1, keepdim=True))
    lp, lse = x - m - lns, m + lns
    p = torch.exp(lp)
    H = -torch.where(p > 0, p * torch.where(p > 0, lp, torch.zeros_like(lp)), torch.zeros_like(p)).sum(1)
    lp = torch.where(none, torch.full_like(lp, -math.inf), lp)
    return lp, torch.where(none[:, 0], 0.0, H), torch.where(none, -math.inf, lse)[:, 0]


def logp_grad(z, ids, dlogp, dentropy, tau):
    """Gradient of sum(dlogp logp + dentropy H); rows with ids < 0 and rows of -inf: 0."""
    lp, H, _ = logp_rows(z, tau)
    T, V = z.shape
    on = torch.ones(T, dtype=torch.bool) if ids is None else (ids >= 0) & (ids < V)
    on = on & ~(z == -math.inf).all(1)
    p = torch.where(on[:, None], torch.exp(lp), 0.0)
    g = torch.zeros_like(p)
    if dlogp is not None:
        hot = torch.zeros_like(p)
        hot[on, ids[on].long()] = 1.0
        g = g + dlogp[:, None] * (hot - p)
    if dentropy is not None:
        ln = torch.where(p > 0, lp, torch.zeros_like(lp))
        g = g - dentropy[:, None] * p * (ln + H[:, None])
    return torch.where(on[:, None], g / tau, 0.0)


def spread(z, tau):
    """Largest distance of a row's finite logits that still have a share, in powers of two; what is further is 0."""
    f = torch.where(torch.isfinite(z), z, torch.full_like(z, math.nan))
    lo, hi = torch.nan_to_num(f, nan=math.inf).amin(1), torch.nan_to_num(f, nan=-math.inf).amax(1)
    r = torch.nan_to_num((hi - lo) / tau * 1.4427, nan=0.0, posinf=0.0, neginf=0.0)
    return r.clamp(min=0, max=160)[:, None]


def logp_bounds(z, tau, lp_at):
    """(logp, entropy, lse) for rows of V: sums in a thread's V / 256 steps, then 40; a term's exponent of
    size R carries R roundings of its own size. The maximum's offset m / tau is rounded at its own size in lse."""
    T, V = z.shape
    R = spread(z, tau)[:, 0]
    n = V / 128 + 64
    lp, H, lse = logp_rows(z, tau)
    step = (n + 8 * R) * U
    at = torch.nan_to_num(lp_at.abs(), posinf=0.0)
    return step + 8 * U * at, step * (2 + H.abs() + math.log(V)), step + 8 * U * torch.nan_to_num(lse.abs(), posinf=0.0)


def logp_grad_bound(z, ids, dlogp, dentropy, tau, dtype):
    T, V = z.shape
    lp, H, _ = logp_rows(z, tau)
    p = torch.exp(lp)
    a = torch.zeros(T, dtype=torch.float64) if dlogp is None else dlogp.abs()
    b = torch.zeros(T, dtype=torch.float64) if dentropy is None else dentropy.abs()
    ln = torch.where(p > 0, lp, torch.zeros_like(lp)).abs()
    R = spread(z, tau)
    n = V / 128 + 64
    size = p * (a[:, None] + b[:, None] * (ln + H.abs()[:, None]))
    got = logp_grad(z, ids, dlogp, dentropy, tau).abs()
    e = (n + 8 * R) * U * (size + b[:, None] * p * math.log(V)) / tau + 8 * U * got
    return e + half_ulp(dtype) * got + TINY


def top(z, K):
    """(ids, logits) by value, equal ones by the lower index; -inf and NaN are none."""
    v = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z) + 0.0
    order = torch.argsort(v, dim=1, descending=True, stable=True)[:, :K]
    val = v.gather(1, order)
    ids = torch.where(val == -math.inf, torch.full_like(order, -1), order)
    if K > z.shape[1]:
        pad = K - z.shape[1]
        ids = torch.cat([ids, ids.new_full((z.shape[0], pad), -1)], 1)
        val = torch.cat([val, val.new_full((z.shape[0], pad), -math.inf)], 1)
    return ids.to(torch.int32), val
