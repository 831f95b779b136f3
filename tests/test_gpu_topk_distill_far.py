"""The distillation loss and gradient of rows with logits far from zero, by value against the 64-bit
form: finite masks over part of a row, whole rows far below or above, all that the list leaves out
masked while the teacher has mass there, masked list entries, in place and not.

Bounds as in operator_ref.distill_bounds, with the exponents that count: distances from the maximum
outside the list and from the row's maximum, up to 200 (beyond, a probability is 0 in both)."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import operator_ref as ref
from test_gpu_topk_distill import DT, make

pytestmark = pytest.mark.gpu

FAR = [-5.0e7, -1.0e10, -1.0e20, -1.0e30, -1.0e38, 5.0e7, 1.0e10, 1.0e20, 1.0e30]
MASKS = [-1.0e8, -1.0e10, -3.0e12, -1.0e20, -1.0e30, -1.0e38, "lowest"]


def softmax_to(z, keep):
    """(softmax over the kept elements, largest exponent that counts)."""
    z = torch.where(keep, z, torch.full_like(z, float("-inf")))
    d = z - z.amax(1, keepdim=True)
    near = d[torch.isfinite(d) & (d > -200)]
    return torch.softmax(z, 1), float(near.abs().max())


def gradient(p, share, outside, ids, teacher, tau, lse, f):
    """From the formula (autograd's logsumexp does not resolve shares of exponents beyond 1e12, even in 64 bits)."""
    valid = ids >= 0
    tl = (teacher / tau).masked_fill(~valid, float("-inf"))
    q = torch.exp(tl - (torch.logsumexp(tl, 1, keepdim=True) if lse is None else lse[:, None]))
    left = (1 - q.sum(1, keepdim=True)).clamp(min=0) if lse is not None else torch.zeros(len(q), 1, dtype=torch.float64)
    S = torch.where(left > 0, torch.ones_like(left), q.sum(1, keepdim=True))
    target = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0).long(), q)
    return f * (S * p - target - torch.where(outside, left * share, torch.zeros_like(p)))


def check(t, in_place=False):
    z, ids, teacher, lse = ref.d(t["z"]), t["ids"].cpu(), ref.d(t["t"]), ref.d(t["lse"])
    tau, scale, dtype = t["tau"], t["scale"], t["z"].dtype
    T, V = z.shape
    loss, rows, _ = ref.distill(z, ids, teacher, tau, lse, None, scale)
    outside = torch.ones(T, V + 1, dtype=torch.bool)
    outside.scatter_(1, torch.where((ids < 0) | (ids >= V), V, ids).long(), False)
    outside = outside[:, :V]
    p, reach = softmax_to(z / tau, torch.ones_like(outside))
    share, reach_out = softmax_to(z / tau, outside)
    R = 1.4427 * max(2 * reach, 2 * reach_out, 2 * float(teacher.abs().max()) / tau, 0.0 if lse is None else float(lse.abs().max())) + 32
    f = scale / tau
    grad = gradient(p, share, outside, ids, teacher, tau, lse, f)
    size = f * (p + (share if lse is not None else 0)) + grad.abs()
    bound = (64 + 4 * R) * ref.U * size + ref.half_ulp(dtype) * grad.abs() + 1e-38
    lp = torch.log_softmax(z / tau, 1)
    listed = torch.where(outside, torch.zeros_like(lp), lp).abs().amax(1)
    rest = torch.logsumexp(torch.where(outside, lp, torch.full_like(lp, float("-inf"))), 1).abs() if lse is not None else 0.0
    row_bound = (64 + 8 * R) * ref.U * (listed + rest + 2 * teacher.abs().amax(1) / tau + 16)
    dz = t["z"].clone() if in_place else torch.empty(T, V, dtype=dtype, device="cuda")
    got, got_rows = dgr.topk_distill(dz if in_place else t["z"], t["ids"], t["t"], tau=tau, teacher_lse=t["lse"], scale=scale, dlogits=dz)
    err = (ref.d(got_rows) - rows).abs()
    assert (err <= row_bound).all(), (got_rows, rows, row_bound)
    assert abs(float(got) - float(loss)) <= scale * float(row_bound.sum()) + 64 * ref.U * scale * float(rows.abs().sum())
    err = (ref.d(dz) - grad).abs()
    assert (err <= bound).all(), (float((err / bound).max()), torch.isnan(dz).any(1), (err > bound).sum(1))
    return got, got_rows, dz


def masks(value, dtype):
    return torch.finfo(DT[dtype]).min if value == "lowest" else value


def unlisted(t):
    T, V = t["z"].shape
    keep = torch.ones(T, V + 1, dtype=torch.bool, device="cuda")
    keep.scatter_(1, torch.where(t["ids"] < 0, V, t["ids"]).long(), False)
    return keep[:, :V]


@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [900, 40000])
def test_masked_parts(V, dtype, tail, value):
    t = make(6, V, 8, dtype, tau=0.9, tail=tail, weights=False)
    at = torch.arange(V, device="cuda")
    for r, closed in enumerate([at >= V // 2, at < V // 2, at % 2 == 1, (at > V // 3) & (at < V - 50), at < V - 20]):
        t["z"][r][closed & unlisted(t)[r]] = masks(value, dtype)
    check(t)


@pytest.mark.parametrize("value", FAR)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [900, 40000])
def test_whole_rows(V, dtype, tail, value):
    t = make(5, V, 8, dtype, tail=tail, weights=False)
    t["z"][0] = value
    t["z"][4] = value                        # the last row too
    if dtype == "fp32" and abs(value) < 1e8:  # a spread that the type still holds: multiples of 4
        t["z"][1] = value + 4.0 * torch.round(t["z"][1])
    else:
        t["z"][1] = value
        t["z"][1, ::3] = value - abs(value) / 2  # a third of it much lower
    t["z"][2, V // 2:] = value               # two levels: one of them far away
    check(t)


@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [900, 40000])
def test_nothing_but_the_list_is_open(V, dtype, value):
    """The gradient outside is -q_r / n each, though the student has no mass there."""
    t = make(4, V, 8, dtype, tau=1.5, tail=True, weights=False)
    t["lse"] += 0.4
    t["z"][unlisted(t)] = masks(value, dtype)
    t["z"][3, 5] = t["z"][3, 5] / 2           # one a little more open than the others
    out = check(t)
    assert bool((out[2][0][unlisted(t)[0]] < 0).all())


@pytest.mark.parametrize("value", [-1.0e10, -1.0e30, "lowest", 1.0e10, 1.0e30])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_far_list_entries(dtype, tail, value):
    t = make(4, 3000, 8, dtype, tau=1.5, tail=tail, weights=False)
    t["ids"][:] = torch.arange(8, dtype=torch.int32, device="cuda") * 301
    t["z"][0, 301] = masks(value, dtype)      # one entry
    t["z"][1, ::301] = masks(value, dtype)    # the whole list
    check(t)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [904, 32768, 40001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place(dtype, V, tail):
    t = make(3, V, 8, dtype, tail=tail, weights=False)
    t["z"][0] = -1.0e30
    t["z"][1, V // 2:] = 1.0e20
    t["z"][2] = torch.finfo(DT[dtype]).min
    out = check(t)
    there = check(t, in_place=True)
    assert all(torch.equal(a, b) for a, b in zip(out, there))


@pytest.mark.parametrize("scale", [0.125, 1.0e-3])
def test_a_loss_in_range_of_rows_whose_sum_is_not(scale):
    t = make(8, 900, 4, "fp32", weights=False)
    t["ids"][:] = torch.arange(4, dtype=torch.int32, device="cuda")
    t["z"][:, :4] = -1.5e38
    t["scale"] = scale
    _, rows, _ = check(t)
    assert bool((rows > 1.0e38).all())


@pytest.mark.parametrize("value", ["lowest", -3.0e38, -1.0e30, 1.0e6, 3.0e38])
@pytest.mark.parametrize("tau", [0.3, 1.0, 1.7])
def test_teachers_far_from_zero(tau, value):
    """Without the teacher's logsumexp its list counts by distances from its own maximum alone."""
    t = make(4, 900, 8, "fp32", tau=tau, weights=False)
    t["ids"][:] = torch.arange(8, dtype=torch.int32, device="cuda") * 7
    near = t["t"].clone()
    t["t"][0] = masks(value, "fp32")
    t["t"][1, 3:] = masks(value, "fp32")
    t["t"][2] = 1.0e6 + torch.round(near[2])
    z, ids, teacher = ref.d(t["z"]), t["ids"].cpu(), ref.d(t["t"])
    teacher = teacher - teacher.amax(1, keepdim=True)  # 64 bits do not resolve a logsumexp's ln K beyond 1e16 either
    loss, rows, grad = ref.distill(z, ids, teacher, tau, None, None, t["scale"])
    dz = torch.empty_like(t["z"])
    got, got_rows = dgr.topk_distill(t["z"], t["ids"], t["t"], tau=tau, scale=t["scale"], dlogits=dz)
    # operator_ref.distill_bounds, with a teacher's distances (up to 200) in the place of its values
    apart = -teacher / tau
    apart = torch.where(apart < 200, apart, torch.zeros_like(apart))
    rel, bound = ref.distill_bounds(z, ids, -apart * tau, tau, None, None, t["scale"], t["z"].dtype, grad)
    size = torch.log_softmax(z / tau, 1).abs().amax(1) + 2 * apart.amax(1) + 16
    assert ((ref.d(got_rows) - rows).abs() <= rel * size).all(), (got_rows, rows)
    assert ((ref.d(dz) - grad).abs() <= bound + 1e-38).all()
