"""Rows of token log probabilities that hold nothing but NaN, or NaN beside masked places: their results and
gradients are NaN; only a row of nothing but -inf has none of its own."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from test_gpu_token_logprobs import INF, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,V,K", [(8, 1, 0), (8, 5, 2), (8, 3000, 0), (8, 3001, 5), (8, 40000, 0), (8, 40000, 20), (1300, 2000, 5)])
def test_rows_without_a_number(T, V, K, dtype):
    """Alone on a CTA, over a cluster, and among many short rows."""
    z, ids = make(T, V, dtype)
    clean = dgr.token_logprobs(z, ids.clamp(min=0), top=K)
    ids.clamp_(min=0)
    z[1] = float("nan")
    z[3] = -INF
    z[3, V // 2] = float("nan")
    z[5] = float("nan")
    z[5, ::2] = -INF
    if V == 1:
        z[5] = float("nan")
    z[6] = -INF
    got = dgr.token_logprobs(z, ids, top=K)
    for k in ("logp", "entropy", "lse"):
        assert got[k][[1, 3, 5]].isnan().all(), k
    assert got["stats"][[1, 3, 5], 1].isnan().all()
    assert float(got["logp"][6]) == -INF == float(got["lse"][6]) and float(got["entropy"][6]) == 0
    if K:
        assert (got["top_ids"][[1, 3, 5, 6]] == -1).all() and (got["top_logits"][[1, 3, 5, 6]] == -INF).all()
    rest = [t for t in range(T) if t not in (1, 3, 5, 6)]
    assert all(torch.equal(got[k][rest], clean[k][rest]) for k in got)
    one = torch.ones(T, device="cuda")
    for which in (dict(dlogp=one), dict(dentropy=one), dict(dlogp=one, dentropy=one)):
        dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], **which)
        assert dz[[1, 3, 5]].isnan().all() and not dz[6].any() and dz[rest].isfinite().all(), which.keys()
    dz = dgr.token_logprobs_backward(z, None, got["stats"], got["entropy"], dentropy=one)
    assert dz[[1, 3, 5]].isnan().all() and not dz[6].any()
    ids[1] = ids[3] = -1  # left out: not read
    got = dgr.token_logprobs(z, ids, top=K)
    dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=one)
    assert not got["logp"][[1, 3]].any() and not dz[[1, 3]].any() and dz[5].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_beside_far_logits(dtype):
    """A row whose scaled maximum leaves the exact integers is read twice; a NaN in it is seen all the same."""
    z, ids = make(8, 3000, dtype)
    ids.clamp_(min=0)
    z[2] = -1e30
    z[2, 9] = float("nan")
    z[4] = torch.finfo(z.dtype).min
    z[4, ::3] = float("nan")
    got = dgr.token_logprobs(z, ids, top=3)
    assert got["logp"][[2, 4]].isnan().all() and got["lse"][[2, 4]].isnan().all()
    dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=torch.ones(8, device="cuda"))
    assert dz[[2, 4]].isnan().all() and dz[[0, 1, 3, 5, 6, 7]].isfinite().all()
