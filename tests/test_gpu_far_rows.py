"""Rows so far apart that their offsets pass 32 bits: the same results as of the rows packed, and nothing between
them written (elements next to each row are held to what they were)."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from test_gpu_gated_ffn import make as make_ffn
from test_gpu_qk_norm_rope import make as make_qk
from test_gpu_token_logprobs import make as make_logits

pytestmark = pytest.mark.gpu


def far(t, ld):
    """t's rows [T, ...] in a buffer with ld elements from a row to the next, 8 known ones behind each."""
    T, n = t.shape[0], t[0].numel()
    assert (T - 1) * ld > 2 ** 31
    buf = torch.empty((T - 1) * ld + n + 8, dtype=t.dtype, device="cuda")
    buf.as_strided((T, n + 8), (ld, 1)).fill_(7.0)
    v = buf.as_strided(t.shape, (ld,) + t.stride()[1:])
    v.copy_(t)
    return v


def behind(v):
    n = v[0].numel()
    return v.as_strided((v.shape[0], 8), (v.stride(0), 1), v.storage_offset() + n)


def held(got, want):
    assert torch.equal(got, want) and (behind(got) == 7.0).all()


@pytest.mark.parametrize("counts,H,F,ld", [([2, 3], 72, 264, 2 ** 29 + 8), ([5500, 4500], 1544, 264, 2 ** 18)])
def test_gated_ffn(counts, H, F, ld):
    t, T = make_ffn(counts, H, F), sum(counts)
    w = dict(offs=t["offs"])
    h, a, b = (torch.empty(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], h=h, gate=a, up=b, **w)
    new = lambda n: far(torch.zeros(T, n, dtype=torch.bfloat16, device="cuda"), ld)  # noqa: E731
    out = dict(h=new(F), gate=new(F), up=new(F))
    dgr.gated_ffn(far(t["x"], ld), t["w_gate"], t["w_up"], **out, **w)
    for k, v in (("h", h), ("gate", a), ("up", b)):
        held(out.pop(k), v)
    want = dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], **w)
    out = dict(dx=new(H), dgate=new(F), dup=new(F))
    dgr.gated_ffn_backward(*(far(t[k], ld) for k in ("dh", "gate", "up")), t["w_gate"], t["w_up"], **out, **w)
    for k in list(out):
        held(out.pop(k), want[k])


@pytest.mark.parametrize("T,D,dtype,ld", [(5, 128, "bf16", 2 ** 29 + 8), (5, 6, "fp32", 2 ** 29 + 2), (3000, 80, "bf16", 2 ** 20)])
def test_qk_norm_rope(T, D, dtype, ld):
    a, (dq, dk) = make_qk(T, 3, 2, D, D, dtype)
    want = dgr.qk_norm_rope(**a)
    back = dgr.qk_norm_rope_backward(dq, dk, **a)
    q = far(a["q"], ld)
    b = dict(a, q=q)
    got = dgr.qk_norm_rope(**b, q_out=far(torch.zeros_like(a["q"]), ld))
    held(got[0], want[0])
    assert torch.equal(got[1], want[1])
    del got
    res = dgr.qk_norm_rope_backward(far(dq, ld), dk, **b, dq=far(torch.zeros_like(a["q"]), ld))
    held(res["dq"], back["dq"])
    assert all(torch.equal(res[k], back[k]) for k in ("dk", "dw_q", "dw_k"))


@pytest.mark.parametrize("T,V,K,dtype,ld", [(5, 5000, 20, "bf16", 2 ** 29 + 8), (3, 40000, 5, "fp32", 2 ** 30 + 4), (700, 2000, 5, "bf16", 2 ** 22)])
def test_token_logprobs(T, V, K, dtype, ld):
    z, ids = make_logits(T, V, dtype)
    want = dgr.token_logprobs(z, ids, top=K)
    one = torch.ones(T, device="cuda")
    dz = dgr.token_logprobs_backward(z, ids, want["stats"], want["entropy"], dlogp=one, dentropy=one)
    y = far(z, ld)
    got = dgr.token_logprobs(y, ids, top=K)
    assert all(torch.equal(got[k], want[k]) for k in want)
    held(dgr.token_logprobs_backward(y, ids, want["stats"], want["entropy"], dlogp=one, dentropy=one, dlogits=far(torch.zeros_like(z), ld)), dz)
    # in place
    held(dgr.token_logprobs_backward(y, ids, want["stats"], want["entropy"], dlogp=one, dentropy=one, dlogits=y), dz)
