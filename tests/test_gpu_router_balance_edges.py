"""The router balance loss with more groups than a CTA has threads."""
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
