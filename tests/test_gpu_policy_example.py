"""The training step of examples/moe_policy.py, which takes the norm and rotation of queries and keys, the gated
experts and the token log probabilities in one run: its gradients against automatic differentiation in 64 bits, two
runs that end in the same bits, and a teacher's lists handed to the distillation."""
import os
import sys

import pytest
import torch

import more_operator_ref as ref
import operator_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_policy as moe  # noqa: E402

pytestmark = pytest.mark.gpu


def loss_64(P, data, chosen):
    """The same step's losses with every intermediate result in 64 bits, for the routing that it chose."""
    T, length, H, D = data["x"].numel(), data["length"], moe.H, moe.D
    cos, sin = (ref.d(t[data["positions"].long().cpu()]) for t in moe.tables(length, "cpu"))
    norm = lambda h, w: operator_ref.block_norm(h, None, None, None, 1.0, w, moe.EPS)[1]  # noqa: E731
    x = P["embed"][data["x"].cpu()]
    packed = norm(x, P["norm1"]) @ P["qkv"]
    q, k, v = packed.split([moe.HEADS * D, moe.KV * D, moe.KV * D], 1)
    q = ref.qk(q.view(T, moe.HEADS, D), P["q_norm"], cos, sin, moe.EPS, False)
    k = ref.qk(k.view(T, moe.KV, D), P["k_norm"], cos, sin, moe.EPS, False)
    h1 = x + moe.attend(q, k, v.view(T, moe.KV, D), length)[0] @ P["proj"]
    u2 = norm(h1, P["norm2"])
    scores = u2 @ P["router"]
    prob = torch.softmax(scores.gather(1, chosen), 1)
    y = torch.zeros(T, H, dtype=torch.float64)
    for s in range(moe.TOPK):
        for e in range(moe.EXPERTS):
            rows = torch.nonzero(chosen[:, s] == e)[:, 0]
            a, b = u2[rows] @ P["w_gate"][e].t(), u2[rows] @ P["w_up"][e].t()
            y = y.index_add(0, rows, prob[rows, s][:, None] * ((ref.activation(a, "silu") * b) @ P["w_down"][e].t()))
    lp, H_, _ = ref.logp_rows(norm(h1 + y, P["norm3"]) @ P["out"], moe.TAU)
    ids = data["ids"].cpu().long()
    on = ids >= 0
    policy = -((ref.d(data["advantage"])[on] * lp[on, ids[on]]).sum() + moe.BONUS * H_[on].sum()) / on.sum()
    return policy, operator_ref.balance(scores, chosen, moe.COEFF)[0]


def routing(P, data):
    """The experts that the step chose, by the same operations."""
    kept = {}
    canonical = moe.dgr.topk_canonicalize

    def keep(*args, **kw):
        kept["out"] = canonical(*args, **kw)
        return kept["out"]

    moe.dgr.topk_canonicalize = keep
    try:
        result = moe.step(P, data)
    finally:
        moe.dgr.topk_canonicalize = canonical
    return result, kept["out"][0].cpu().long()


def test_gradients():
    P, data = moe.parameters(3), moe.batch(3, 40, 5)
    (loss, balance, got), chosen = routing(P, data)
    W = {k: v.to(torch.bfloat16).cpu().double().requires_grad_() for k, v in P.items()}
    want, want_balance = loss_64(W, data, chosen)
    grads = torch.autograd.grad(want + want_balance, list(W.values()))
    want, want_balance = want.detach(), want_balance.detach()
    # rounded logits (2^-8 of up to 4 each) over about a hundred tokens of either sign, and the sum's own size
    assert abs(float(loss) - float(want)) <= 0.02 * (1 + abs(float(want)))
    assert abs(float(balance) - float(want_balance)) <= 0.01 * float(want_balance)
    # up to twenty roundings to bf16 (2^-8 each, mostly independent) lie between the loss and a gradient: 1 to 2 % of
    # its norm, 5 % at most
    for (k, w), g in zip(W.items(), grads):
        off = float((ref.d(got[k]) - g).norm() / g.norm())
        assert off <= 0.05, (k, off)


def test_reproducible():
    a, P = moe.train(3, sequences=4, length=32)
    b, Q = moe.train(3, sequences=4, length=32)
    assert a == b and all(torch.equal(P[k], Q[k]) for k in P)


def test_teacher_lists():
    g = torch.Generator().manual_seed(4)
    teacher, student = (2 * torch.randn(20, moe.VOCAB, generator=g) for _ in range(2))
    ids, logits, lse = moe.teacher_lists(teacher.cuda(), 1.5)
    _, rows = moe.dgr.topk_distill(student.cuda(), ids, logits, tau=1.5, teacher_lse=lse)
    best = teacher.double().topk(moe.LIST, dim=1)
    want = operator_ref.distill_rows(student.double(), best.indices, best.values, 1.5, torch.logsumexp(teacher.double() / 1.5, 1))
    assert ((ref.d(rows) - want).abs() <= 1e-5 * (1 + want.abs())).all()
