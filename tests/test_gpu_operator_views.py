"""Tensors that lie between one another's rows or heads in one buffer, without an element in common: the calls take
them, write what is theirs, and give the bits that tensors of their own give."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from test_gpu_qk_norm_rope import DT, EPS, make as make_qk

pytestmark = pytest.mark.gpu


def alternating(t, dy, kinds=3):
    """q, k (and a third) head by head in one row: [T, heads, kinds, D]; outputs in place."""
    T, n, D = t["q"].shape
    row = torch.full((T, n, kinds, D), 5.0, dtype=t["q"].dtype, device="cuda")
    row[:, :, 0], row[:, :, 1] = t["q"], t["k"]
    return row


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,n,D,R", [(21, 6, 64, 32), (1, 4, 128, 128), (5, 1, 64, 64), (7, 3, 42, 20)])
def test_heads_of_queries_and_keys_in_turn(T, n, D, R, dtype):
    t, dy = make_qk(T, n, n, D, R, dtype)
    want = dgr.qk_norm_rope(**t, eps=EPS)
    back = dgr.qk_norm_rope_backward(*dy, **t, eps=EPS)
    row = alternating(t, dy)
    u = dict(t, q=row[:, :, 0], k=row[:, :, 1])
    got = dgr.qk_norm_rope_backward(*dy, **u, eps=EPS)
    assert all(torch.equal(got[k], back[k]) for k in back)
    grad = torch.full_like(row, 7.0)  # the gradients in a row like it, beside those of a third kind
    got = dgr.qk_norm_rope_backward(*dy, **u, eps=EPS, dq=grad[:, :, 0], dk=grad[:, :, 1])
    assert all(torch.equal(got[k], back[k]) for k in back) and (grad[:, :, 2] == 7).all()
    grad[:, :, 0], grad[:, :, 1] = dy[0], dy[1]  # and in place of the outputs' gradients
    got = dgr.qk_norm_rope_backward(grad[:, :, 0], grad[:, :, 1], **u, eps=EPS, dq=grad[:, :, 0], dk=grad[:, :, 1])
    assert all(torch.equal(got[k], back[k]) for k in back) and (grad[:, :, 2] == 7).all()
    y = dgr.qk_norm_rope(**u, eps=EPS, q_out=row[:, :, 0], k_out=row[:, :, 1])
    assert all(torch.equal(a, b) for a, b in zip(y, want)) and (row[:, :, 2] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_heads_before_tokens_in_turn(dtype):
    """[heads, kinds, T, D], and fewer keys than queries between them."""
    T, A, B, D = 19, 4, 4, 64
    t, dy = make_qk(T, A, B, D, D, dtype)
    want = dgr.qk_norm_rope(**t, eps=EPS)
    buf = torch.full((A, 2, T, D), 5.0, dtype=DT[dtype], device="cuda")
    views = [buf[:, i].transpose(0, 1) for i in range(2)]
    views[0].copy_(t["q"]), views[1].copy_(t["k"])
    got = dgr.qk_norm_rope(**dict(t, q=views[0], k=views[1]), eps=EPS, q_out=views[0], k_out=views[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    t, dy = make_qk(T, 6, 2, D, D, dtype)
    want = dgr.qk_norm_rope(**t, eps=EPS)
    row = torch.full((T, 6, 2, D), 5.0, dtype=DT[dtype], device="cuda")
    row[:, :, 0], row[:, 3:5, 1] = t["q"], t["k"]
    u = dict(t, q=row[:, :, 0], k=row[:, 3:5, 1])
    got = dgr.qk_norm_rope(**u, eps=EPS, q_out=u["q"], k_out=u["k"])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (row[:, :3, 1] == 5).all() and (row[:, 5:, 1] == 5).all()
