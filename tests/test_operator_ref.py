"""The 64-bit references of the operators' tests, held against finite differences.

Central differences in 64 bits with a step of 1e-5: their error is of the order of the step squared
(1e-10) plus 2^-53 / step (1e-11) times the values, well below the 1e-6 asked for.
"""
import math

import pytest
import torch

import operator_ref as ref

STEP, TOL = 1e-5, 1e-6


def differences(f, x):
    g = torch.zeros_like(x)
    flat = x.reshape(-1)
    for i in range(flat.numel()):
        old = flat[i].item()
        flat[i] = old + STEP
        up = float(f(x))
        flat[i] = old - STEP
        down = float(f(x))
        flat[i] = old
        g.reshape(-1)[i] = (up - down) / (2 * STEP)
    return g


def close(got, want):
    assert torch.allclose(got, want, rtol=TOL, atol=TOL), float((got - want).abs().max())


def rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance(score):
    g = torch.Generator().manual_seed(1)
    x, ids = rand(g, 9, 5), torch.randint(-1, 5, (9, 2), generator=g)
    offs, mask = [0, 3, 3, 9], torch.tensor([1, 1, 0, 1, 1, 1, 0, 1, 1])
    f = lambda v: ref.balance(v, ids, 0.3, offs, mask, score)[0]  # noqa: E731
    v = x.clone().requires_grad_()
    grad = torch.autograd.grad(f(v), v)[0]
    close(grad, differences(f, x.clone()))
    # the closed form that the kernels use
    loss, counts, tokens = ref.balance(x, ids, 0.3, offs, mask, score)
    p = ref.balance_scores(x, score)
    for t in range(9):
        s = 0 if t < 3 else 2
        a = 0.3 * 5 / (3 * 2 * int(tokens[s]) ** 2)
        c = counts[s].double()
        want = a * p[t] * (c - (c * p[t]).sum()) * (mask[t] != 0)
        if score == "sigmoid":
            want = want * (1 - torch.sigmoid(x[t]))
        close(grad[t], want)
    assert tokens.tolist() == [2, 0, 5] and float(loss) > 0


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm(gate, post):
    g = torch.Generator().manual_seed(2)
    T, H, a, eps = 3, 6, 0.7, 1e-2
    x, y, dh, du = (rand(g, T, H) for _ in range(4))
    w1 = rand(g, H) if post else None
    w2 = rand(g, H)
    gt = {"none": None, "channel": rand(g, H), "token": rand(g, T, 1)}[gate]

    def total(**new):
        at = {**dict(x=x, y=y, w_post=w1, gate=gt, w_pre=w2), **new}
        h, u = ref.block_norm(at["x"], at["y"], at["w_post"], at["gate"], a, at["w_pre"], eps)
        return (h * dh).sum() + (u * du).sum()

    h, _ = ref.block_norm(x, y, w1, gt, a, w2, eps)
    got = ref.block_norm_grads(h, y, dh, du, w1, gt, a, w2, eps)
    for name, key, value in (("dx", "x", x), ("dy", "y", y), ("dw_post", "w_post", w1), ("dgate", "gate", gt),
                             ("dw_pre", "w_pre", w2)):
        if value is not None:
            close(got[name], differences(lambda v: total(**{key: v}), value.clone()))


@pytest.mark.parametrize("tail", [False, True])
def test_distill(tail):
    g = torch.Generator().manual_seed(3)
    T, V, K, tau = 5, 7, 3, 1.7
    z, full = 2 * rand(g, T, V), 2 * rand(g, T, V)
    top = full.topk(K, dim=1)
    ids = top.indices.clone()
    ids[1, 2] = -1
    ids[2, :] = -1
    ids[3, 2] = ids[3, 0]  # an id twice
    lse = torch.logsumexp(full / tau, 1) if tail else None
    w = torch.tensor([1.0, 0.5, 1.0, 2.0, 0.0], dtype=torch.float64)
    f = lambda v: ref.distill(v, ids, top.values, tau, lse, w, 0.4)[0]  # noqa: E731
    loss, rows, grad = ref.distill(z, ids, top.values, tau, lse, w, 0.4)
    close(grad, differences(f, z.clone()))
    assert float(rows[2]) == 0.0 and float(rows[4]) == 0.0 and not bool(grad[2].any()) and not bool(grad[4].any())
    # the closed form that the kernels use
    for t in (0, 1, 3):
        p = torch.softmax(z[t] / tau, 0)
        ok = ids[t] >= 0
        tl = torch.where(ok, top.values[t] / tau, -math.inf)
        q = torch.exp(tl - (torch.logsumexp(tl, 0) if lse is None else lse[t]))
        want = p.clone()
        if tail:
            inside = torch.zeros(V, dtype=torch.bool)
            inside[ids[t][ok]] = True
            want = torch.where(inside, p, p * (1 - max(0.0, 1 - float(q.sum())) / p[~inside].sum()))
        want.scatter_add_(0, ids[t].clamp(min=0), -q)
        close(grad[t], want * 0.4 * w[t] / tau)
