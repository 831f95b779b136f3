"""The router balance loss with more groups than a CTA has threads, of rows of logits far from zero, and with one
workspace for calls of other sizes."""
import numpy as np
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import operator_ref as ref
from gpu_util import bits
from test_gpu_router_balance import COEFF, _call, make

pytestmark = pytest.mark.gpu


def cuts_of(G, N, seed):
    return sorted([0, N] + np.random.RandomState(seed).randint(0, N + 1, G - 1).tolist())


@pytest.mark.parametrize("G", [513, 700, 1024])
@pytest.mark.parametrize("dtype,E", [("fp32", 520), ("bf16", 1024), ("bf16", 601)])
def test_more_groups_than_a_cta_has_threads(dtype, E, G):
    """Rows of more than 16 logits a lane run on CTAs of 512 threads, which take the offsets in two rounds."""
    t = make(1500, E, 2, dtype, offs=cuts_of(G, 1500, G))
    loss, counts, tokens = dgr.router_balance(t["x"], t["ids"], COEFF, offs=t["offs"])
    wl, wc, wt = ref.balance(ref.d(t["x"]), t["ids"].cpu(), COEFF, t["offs"].tolist())
    assert torch.equal(counts.cpu().long(), wc) and torch.equal(tokens.cpu().long(), wt)
    # as in test_gpu_router_balance.check, and the sum over groups: at most 2 of a thread's, then lanes and warps
    rel = (64 + 4 * ref.finite_range(ref.d(t["x"])) + 2 * (1500 // 256 + 8) + E // 32 + 2 + 5 + 16) * ref.U
    assert abs(float(loss) - float(wl)) <= rel * float(wl)
    base = bits(_call(t))
    for _ in range(30):
        assert (bits(_call(t)) == base).all()


def near_range(x):
    """Largest distance of a logit that counts from its row's maximum (in powers of two): beyond 200 a
    probability is 0 in both."""
    d = x.amax(1, keepdim=True) - x
    d = d[torch.isfinite(d) & (d < 200)]
    return 1.4427 * float(d.max())


@pytest.mark.parametrize("value", [-5.0e7, -1.0e10, -1.0e20, -1.0e30, 5.0e7, 1.0e10, 1.0e20, 1.0e30])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [16, 60, 128, 33])
def test_rows_far_from_zero(E, dtype, score, value):
    t = make(40, E, 2, dtype)
    t["x"][1] = value
    t["x"][2, : E // 2] = value
    t["x"][3] = value
    t["x"][3, 5] = value + abs(value) / 2
    t["x"][39] = value
    if dtype == "fp32" and abs(value) < 1e8:
        t["x"][4] = value + 4.0 * torch.round(t["x"][4])
    loss, counts, tokens = dgr.router_balance(t["x"], t["ids"], COEFF, score=score)
    got = dgr.router_balance_backward(t["x"], counts, tokens, 2, COEFF, score=score)
    v = ref.d(t["x"]).requires_grad_()
    wl, wc, _ = ref.balance(v, t["ids"].cpu(), COEFF, score=score)
    want = torch.autograd.grad(wl, v)[0]
    x = v.detach() if score == "softmax" else torch.nn.functional.logsigmoid(v.detach())
    rel = (64 + 4 * near_range(x) + 16 + E // 32) * ref.U  # as in test_gpu_router_balance.check, for N < 256
    assert abs(float(loss) - float(wl)) <= rel * float(wl)
    p, c = ref.balance_scores(v.detach(), score), wc[0].double()
    a = COEFF * E / (2 * 40 ** 2)
    bound = a * rel * p * (c + (p * c).sum(1, keepdim=True)) + ref.half_ulp(t["x"].dtype) * want.abs() + 1e-38
    err = (ref.d(got) - want).abs()
    assert (err <= bound).all(), (float((err / bound).max()), torch.isnan(got).any(1).nonzero())


def test_one_workspace_for_calls_of_other_sizes():
    """The workspace is zeroed once and then serves calls of any sizes that fit it."""
    # groups of one tile and of several, more than 64 groups after fewer and fewer after more
    sizes = [(3000, 64, 1), (30000, 128, 200), (900, 16, 300), (60000, 64, 90), (64, 4, 1), (2000, 8, 1024), (20000, 64, 33),
             (40000, 32, 130), (700, 520, 600), (3000, 64, 1)]
    ws = dgr.workspace(max(dgr.router_balance_workspace_bytes(*s) for s in sizes))
    for N, E, G in sizes:
        t = make(N, E, 4, "fp32", offs=None if G == 1 else cuts_of(G, N, G), masked=True)
        same = dict(offs=t["offs"], mask=t["mask"])
        want = dgr.router_balance(t["x"], t["ids"], COEFF, **same)
        out = dict(loss=torch.full((1,), -3.0, device="cuda"), counts=torch.full((G, E), -3, dtype=torch.int32, device="cuda"),
                   tokens=torch.full((G,), -3, dtype=torch.int32, device="cuda"))
        for _ in range(2):
            got = dgr.router_balance(t["x"], t["ids"], COEFF, ws=ws, **same, **out)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (N, E, G)
