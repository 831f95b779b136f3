"""The order of the distillation's sums: with a gradient and without, and from run to run where ids come
twice."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from gpu_util import bits
from test_gpu_topk_distill import DT, _call

pytestmark = pytest.mark.gpu


def rows_of(T, V, K, dtype, tail, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + V + K)
    z = (2.0 * torch.randn(T, V, generator=g, device="cuda")).to(DT[dtype])
    full = z.float() * 0.7 + 2.0 * torch.randn(T, V, generator=g, device="cuda")
    top = full.topk(K, dim=1)
    lse = torch.logsumexp(full, 1) if tail else None
    return dict(z=z, ids=top.indices.to(torch.int32), t=top.values.contiguous(), lse=lse, w=None, tau=1.0, scale=0.3)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,V,dtype", [(160, 5000, "fp32"), (310, 20000, "bf16"), (700, 20001, "fp32"), (160, 65536, "bf16"),
                                       (200, 32768, "fp32"), (1000, 50001, "bf16"), (152, 4097, "bf16")])
def test_losses_have_the_same_bits_with_a_gradient_and_without(T, V, dtype, tail):
    """Rows of up to 128 KB."""
    t = rows_of(T, V, 40, dtype, tail)
    same = dict(teacher_lse=t["lse"], scale=t["scale"])
    a = dgr.topk_distill(t["z"], t["ids"], t["t"], **same)
    dz = torch.empty_like(t["z"])
    b = dgr.topk_distill(t["z"], t["ids"], t["t"], dlogits=dz, **same)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), int((a[1] != b[1]).sum())
    assert torch.equal(dgr.topk_distill_backward(t["z"], t["ids"], t["t"], **same), dz)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,V,dtype", [(160, 131072, "bf16"), (700, 131072, "bf16"), (200, 40000, "fp32"), (152, 150001, "fp32")])
def test_longer_rows_keep_their_bits_in_either_form(T, V, dtype, tail):
    """Rows beyond 128 KB lie over more CTAs with a gradient than without one: other orders, each of them fixed,
    and losses within each other's rounding."""
    t = rows_of(T, V, 40, dtype, tail)
    same = dict(teacher_lse=t["lse"], scale=t["scale"])
    a = dgr.topk_distill(t["z"], t["ids"], t["t"], **same)
    dz = torch.empty_like(t["z"])
    b = dgr.topk_distill(t["z"], t["ids"], t["t"], dlogits=dz, **same)
    assert torch.equal(dgr.topk_distill_backward(t["z"], t["ids"], t["t"], **same), dz)
    for _ in range(4):
        c, d = dgr.topk_distill(t["z"], t["ids"], t["t"], **same), dgr.topk_distill(t["z"], t["ids"], t["t"], dlogits=dz, **same)
        assert all(torch.equal(x, y) for x, y in zip(a + b, c + d))
    # twice the bound of operator_ref.distill_bounds: 64 + 8 R roundings of the sizes met
    z, top = t["z"].float(), t["t"].abs().max()
    reach = 1.4427 * max(2 * float(z.abs().max()), 2 * float(top), 0.0 if t["lse"] is None else float(t["lse"].max())) + 32
    size = torch.log_softmax(z, 1).abs().amax(1) + 2 * top + 16
    assert ((a[1] - b[1]).abs() <= 2 * (64 + 8 * reach) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("V", [3000, 20000])
@pytest.mark.parametrize("tail", [False, True])
def test_ids_that_come_twice_give_the_same_bits_every_time(V, tail):
    t = rows_of(600, V, 512, "fp32", tail)
    t["ids"][:, 256:] = t["ids"][:, :256].flip(1)  # the copies lie in other warps
    t["z"] *= 3.0
    base = bits(_call(t))
    for _ in range(20):
        assert (bits(_call(t)) == base).all()
