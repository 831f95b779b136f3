"""Matrices that lie side by side in the rows of one buffer: the gated feed-forward and the token log probabilities
take them, write what is theirs, and give the bits that matrices of their own give."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from test_gpu_gated_ffn import BF, make as make_ffn
from test_gpu_token_logprobs import DT, make as make_logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,H,F", [([1], 64, 72), ([130, 7, 0, 64], 264, 200)])
def test_both_products_in_one_row(counts, H, F):
    """gate beside up, as one projection of both leaves them, h behind them; their gradients over them."""
    t, T = make_ffn(counts, H, F), sum(counts)
    alone = {k: torch.empty(T, F, dtype=BF, device="cuda") for k in ("h", "gate", "up")}
    dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], **alone)
    row = torch.full((T, 3 * F + 8), 5.0, dtype=BF, device="cuda")
    part = {k: row[:, i * F:(i + 1) * F] for i, k in enumerate(("gate", "up", "h"))}
    dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], **part)
    assert all(torch.equal(part[k], alone[k]) for k in alone) and (row[:, 3 * F:] == 5).all()
    back = dgr.gated_ffn_backward(t["dh"], alone["gate"], alone["up"], t["w_gate"], t["w_up"], offs=t["offs"])
    wide = torch.full((T, 2 * F), 7.0, dtype=BF, device="cuda")
    got = dgr.gated_ffn_backward(t["dh"], part["gate"], part["up"], t["w_gate"], t["w_up"], offs=t["offs"], dgate=wide[:, :F], dup=wide[:, F:])
    assert all(torch.equal(got[k], back[k]) for k in back)
    got = dgr.gated_ffn_backward(t["dh"], part["gate"], part["up"], t["w_gate"], t["w_up"], offs=t["offs"], dgate=part["gate"], dup=part["up"])
    assert all(torch.equal(got[k], back[k]) for k in back) and torch.equal(part["h"], alone["h"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_logits_gradient_beside_them(dtype):
    z, ids = make_logits(6, 999, dtype)
    one = torch.ones(6, device="cuda")
    got = dgr.token_logprobs(z, ids)
    want = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=one)
    row = torch.full((6, 2 * 999 + 3), 5.0, dtype=DT[dtype], device="cuda")
    row[:, 2:1001] = z
    dz = dgr.token_logprobs_backward(row[:, 2:1001], ids, got["stats"], got["entropy"], dlogp=one, dlogits=row[:, 1001:2000])
    assert torch.equal(dz, want) and torch.equal(row[:, 2:1001], z) and (row[:, :2] == 5).all() and (row[:, 2000:] == 5).all()
