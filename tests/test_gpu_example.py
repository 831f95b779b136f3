"""The training step of examples/moe_distillation.py: its gradients against automatic differentiation
in 64 bits, its progress, and two runs that end in the same bits."""
import os
import sys

import pytest
import torch

import operator_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_distillation as moe  # noqa: E402

pytestmark = pytest.mark.gpu


def loss_64(P, data, ids):
    """The same step's two losses with every intermediate result in 64 bits, for the routing that it chose."""
    T = data["x"].numel()
    x = P["embed"][data["x"].cpu()]
    _, u0 = ref.block_norm(x, None, None, None, 1.0, P["norm"], moe.EPS)
    scores = u0 @ P["router"]
    prob = torch.softmax(scores.gather(1, ids), 1)
    y = torch.zeros(T, moe.H, dtype=torch.float64)
    for k in range(moe.TOPK):
        for e in range(moe.EXPERTS):
            rows = torch.nonzero(ids[:, k] == e)[:, 0]
            y = y.index_add(0, rows, prob[rows, k][:, None] * (u0[rows] @ P["experts"][e].t() + P["bias"][e]))
    _, u = ref.block_norm(x, y, P["post"], P["gate"], moe.RES_SCALE, P["pre"], moe.EPS)
    rows = ref.distill_rows(u @ P["out"], data["ids"].cpu(), ref.d(data["teacher"]), moe.TAU, ref.d(data["lse"]), ref.d(data["weights"]))
    distillation = moe.TAU ** 2 / T * (ref.d(data["weights"]) * rows).sum()
    return distillation, ref.balance(scores, ids, moe.COEFF)[0]


def test_gradients():
    P, data = moe.parameters(3), moe.batch(200, 5)
    loss, balance, got = moe.step(P, data)
    W = {k: v.to(torch.bfloat16).cpu().double().requires_grad_() for k, v in P.items()}
    # the routing that the step chose: from scores that differ by roundings only
    bf = {k: v.to(torch.bfloat16) for k, v in P.items()}
    _, u0 = moe.dgr.block_norm(bf["embed"][data["x"]], w_pre=bf["norm"], eps=moe.EPS)
    ids = (u0.float() @ bf["router"].float()).topk(moe.TOPK, dim=1).indices.cpu()
    ids = torch.sort(ids, dim=1).values
    want, want_balance = loss_64(W, data, ids)
    total = want + want_balance
    want, want_balance = want.detach(), want_balance.detach()
    assert abs(float(loss) - float(want)) <= 0.01 * float(want)
    assert abs(float(balance) - float(want_balance)) <= 0.01 * float(want_balance)
    grads = torch.autograd.grad(total, list(W.values()))
    # about ten roundings to bf16 (2^-8 each, mostly independent) lie between loss and gradient: 1 to 2 % of a
    # gradient's norm, 4 % at most
    for (k, w), g in zip(W.items(), grads):
        off = float((ref.d(got[k]) - g).norm() / g.norm())
        assert off <= 0.04, (k, off)


def test_training_makes_progress_and_is_reproducible():
    losses, P = moe.train(12, tokens=512)
    assert losses[-1][0] < 0.9 * losses[0][0], losses
    again, Q = moe.train(12, tokens=512)
    assert again == losses and all(torch.equal(P[k], Q[k]) for k in P)
