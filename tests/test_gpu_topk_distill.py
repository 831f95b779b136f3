"""GPU results of the distillation loss and its gradient against the 64-bit form.

Vocabularies from one token to long odd ones, lists that are short, empty, padded, doubled or as
long as the vocabulary, with and without the teacher's mass outside the list, temperatures, weights
of zero over rows of NaN, -inf logits, strided, misaligned and in-place rows, few and many rows, no
rows, launch schedules, replays, other streams.
"""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import operator_ref as ref
from gpu_util import assert_replays_identical, bits
from test_gpu_schedule import SCHEDULES, schedule

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(T, V, K, dtype, tau=1.0, tail=False, pad=0, weights=True, seed=0):
    g = torch.Generator().manual_seed(seed + 13 * T + V + K)
    buf = torch.full((T, V + pad), float("nan"), dtype=DT[dtype])
    z = 2.0 * torch.randn(T, V, generator=g)
    buf[:, :V] = z.to(DT[dtype])
    full = 0.7 * z + 2.0 * torch.randn(T, V, generator=g)
    top = full.topk(K, dim=1)
    ids = top.indices.to(torch.int32)
    ids[torch.rand(T, K, generator=g) < 0.1] = -1
    lse = torch.logsumexp(full.double() / tau, 1).float() if tail else None
    w = (torch.rand(T, generator=g) * (torch.rand(T, generator=g) > 0.2)) if weights else None
    cuda = lambda v: None if v is None else v.cuda()  # noqa: E731
    return dict(z=buf.cuda()[:, :V], ids=ids.cuda(), t=top.values.contiguous().cuda(), lse=cuda(lse), w=cuda(w), tau=tau,
                scale=0.31)


def want_of(t):
    z = ref.d(t["z"])
    if t["w"] is not None:
        z[ref.d(t["w"]) == 0] = 0.0  # such a row is not read
    args = [z, t["ids"].cpu(), ref.d(t["t"]), t["tau"], ref.d(t["lse"]), ref.d(t["w"]), t["scale"]]
    loss, rows, grad = ref.distill(*args)
    rel, bound = ref.distill_bounds(*args, t["z"].dtype, grad)
    # a row's loss: each term q (ln q - ln p) with its own size; they are bounded by ln of the
    # smallest p and q met
    T = z.shape[0]
    lp = torch.log_softmax(torch.nan_to_num(z, nan=0.0) / t["tau"], 1)
    lp = torch.where(torch.isfinite(lp), lp, torch.zeros_like(lp))
    size = lp.abs().amax(1) + 2 * torch.nan_to_num(ref.d(t["t"]), neginf=0.0).abs().amax(1) / t["tau"] + 16
    return loss, rows, grad, rel * size, bound


def check(t, mode="both", **kw):
    loss, rows, grad, row_bound, bound = want_of(t)
    same = dict(tau=t["tau"], teacher_lse=t["lse"], weights=t["w"], scale=t["scale"])
    out = {}
    if mode == "both":
        kw.setdefault("dlogits", torch.full(t["z"].shape, 3.0, dtype=t["z"].dtype, device="cuda"))
    if mode != "backward":
        gl, gr = dgr.topk_distill(t["z"], t["ids"], t["t"], **same, **kw)
        err = (ref.d(gr) - rows).abs()
        assert (err <= row_bound).all(), (float((err / row_bound).max()), gr, rows)
        w = torch.ones_like(rows) if t["w"] is None else ref.d(t["w"])
        lb = t["scale"] * ((w * row_bound).sum() + (64 + len(rows) // 100) * ref.U * (w * rows).abs().sum())
        assert abs(float(gl) - float(loss)) <= lb + 1e-40, (float(gl), float(loss))
        out.update(loss=gl, rows=gr)
    got = kw.get("dlogits")
    if mode == "backward":
        got = dgr.topk_distill_backward(t["z"], t["ids"], t["t"], **same, **kw)
    if got is not None:
        err = (ref.d(got) - grad).abs()
        assert (err <= bound + 1e-40).all(), float((err / (bound + 1e-40)).max())
        out["dz"] = got
    return out


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (2, 3, 2), (3, 9, 9), (5, 100, 7), (4, 1000, 64), (3, 4097, 20), (2, 16384, 128),
                                   (3, 20011, 50), (1, 50001, 33), (2, 131072, 64), (40, 257, 16)])
def test_sizes(T, V, K, dtype, tail):
    t = make(T, V, K, dtype, tau=1.3, tail=tail)
    a = check(t, "both")
    b = check(t, "forward")
    c = check(t, "backward")
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["rows"], b["rows"]) and torch.equal(a["dz"], c["dz"])


@pytest.mark.parametrize("tau", [0.25, 1.0, 4.0, 20.0])
@pytest.mark.parametrize("tail", [False, True])
def test_temperatures(tau, tail):
    check(make(6, 3000, 40, "fp32", tau=tau, tail=tail))


@pytest.mark.parametrize("tail", [False, True])
def test_long_lists(tail):
    check(make(3, 3000, 1024, "bf16", tail=tail))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_special_lists(dtype, tail):
    t = make(8, 700, 12, dtype, tail=tail, weights=False)
    t["ids"][0] = -1                        # nothing taught
    t["ids"][1, 1:] = -1                    # one entry
    t["ids"][2, 3] = t["ids"][2, 7] = t["ids"][2, 5] = 11  # an id three times
    t["t"][3] = float("-inf")               # the teacher gives its list nothing
    t["t"][4, 2:5] = float("-inf")
    t["t"][5] = -3.0e38                     # the type's lowest values
    t["ids"][6] = t["ids"][6].flip(0)
    if tail:
        t["lse"][5] = 50.0
    out = check(t)
    assert not bool(out["dz"][0].any()) and float(out["rows"][0]) == 0.0


def test_list_as_long_as_the_vocabulary():
    t = make(4, 16, 16, "fp32", tail=True, weights=False)
    t["ids"] = torch.arange(16, dtype=torch.int32, device="cuda").repeat(4, 1)
    check(t)


@pytest.mark.parametrize("tail", [False, True])
def test_infinities(tail):
    t = make(6, 900, 8, "bf16", tail=tail, weights=False)
    keep = torch.zeros(900, dtype=torch.bool, device="cuda")
    for r in range(6):
        keep[:] = False
        keep[t["ids"][r][t["ids"][r] >= 0].long()] = True
        if r == 0:
            t["z"][r][~keep] = float("-inf")   # no mass outside the list
        elif r < 4:
            closed = (torch.arange(900, device="cuda") % 3 == 0) & ~keep
            t["z"][r][closed] = float("-inf")  # a padded vocabulary
    out = check(t)
    assert bool(torch.isfinite(out["dz"]).all())


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [900, 20000])
def test_lowest_and_largest_values(V, dtype, tail):
    t = make(6, V, 8, dtype, tau=0.7, tail=tail, weights=False)
    low = torch.finfo(DT[dtype]).min
    t["ids"][:, 0] = 3
    closed = torch.arange(V, device="cuda") >= V // 2  # a mask of the type's lowest value
    closed[t["ids"][t["ids"] >= 0].long()] = False
    t["z"][0][closed] = low
    t["z"][1][:] = low                  # a row that the mask leaves nothing of
    t["z"][2][:] = 2.5e38               # k times the maximum is out of range
    t["z"][2][3] = 2.5e38
    t["z"][3][:] = -2.0e38
    t["z"][3][closed] = low
    t["z"][4] += 1000.0
    z = ref.d(t["z"])
    if not tail:
        # p is uniform over the largest logits; the bound's exponents would be those of the values themselves
        same = dict(tau=t["tau"], scale=t["scale"])
        dz = torch.empty_like(t["z"])
        loss, rows = dgr.topk_distill(t["z"], t["ids"], t["t"], dlogits=dz, **same)
        _, want_rows, want = ref.distill(z, t["ids"].cpu(), ref.d(t["t"]), t["tau"], None, None, t["scale"])
        eps = 2 * ref.half_ulp(t["z"].dtype) + 1e-5
        for r in (0, 1, 2, 3):
            assert bool(torch.isfinite(dz[r]).all()) and abs(float(rows[r]) - float(want_rows[r])) <= 1e-5 * (1 + abs(float(want_rows[r]))), r
            assert float((ref.d(dz[r]) - want[r]).norm()) <= eps * float(want[r].norm()), r
    else:
        dz = torch.empty_like(t["z"])
        loss, rows = dgr.topk_distill(t["z"], t["ids"], t["t"], tau=t["tau"], teacher_lse=t["lse"], scale=t["scale"], dlogits=dz)
        assert bool(torch.isfinite(dz).all()) and bool(torch.isfinite(rows[[0, 1, 2, 3]]).all())


def test_little_mass_outside_the_list():
    t = make(3, 5000, 4, "fp32", tail=True, weights=False)
    t["ids"] = torch.tensor([[1, 2, 3, 4]] * 3, dtype=torch.int32, device="cuda")
    t["z"][:, 1:5] += torch.tensor([[60.0], [120.0], [200.0]], device="cuda")  # p_r down to e^-190
    out = check(t)
    assert bool(torch.isfinite(out["dz"]).all()) and bool(torch.isfinite(out["rows"]).all())


def test_rows_without_weight_are_not_read():
    t = make(10, 2000, 16, "bf16", tail=True)
    t["w"][3] = t["w"][9] = 0.0
    clean = check(t)
    t["z"][3] = float("nan")
    t["t"][9] = float("nan")
    t["lse"][9] = float("nan")
    t["ids"][3] = -7
    got = dgr.topk_distill(t["z"], t["ids"], t["t"], tau=t["tau"], teacher_lse=t["lse"], weights=t["w"], scale=t["scale"],
                           dlogits=torch.empty_like(t["z"]))
    assert torch.equal(got[0], clean["loss"]) and torch.equal(got[1], clean["rows"])
    assert float(got[1][3]) == 0.0


def test_nan_logit_stays_in_its_row():
    t = make(5, 3000, 16, "fp32", weights=False)
    clean = check(t)
    t["z"][2, 1234] = float("nan")
    dz = torch.empty_like(t["z"])
    _, rows = dgr.topk_distill(t["z"], t["ids"], t["t"], tau=t["tau"], scale=t["scale"], dlogits=dz)
    keep = torch.arange(5, device="cuda") != 2
    assert torch.equal(dz[keep], clean["dz"][keep]) and torch.equal(rows[keep], clean["rows"][keep])
    assert bool(torch.isnan(rows[2])) and bool(torch.isnan(dz[2]).all())


def test_ids_beyond_the_vocabulary_are_recorded():
    t = make(4, 300, 8, "fp32", weights=False)
    want = check(t)
    ws = dgr.workspace(dgr.topk_distill_workspace_bytes(4))
    dz = torch.empty_like(t["z"])
    loss, rows = dgr.topk_distill(t["z"], torch.where(t["ids"] < 0, 300, t["ids"]), t["t"], tau=t["tau"], scale=t["scale"],
                                  dlogits=dz, ws=ws)
    assert torch.equal(loss, want["loss"]) and torch.equal(dz, want["dz"])
    assert dgr.read_device_status(ws) == 1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,pad", [(5000, 8), (5001, 7), (5001, 2), (333, 1), (20001, 3)])
def test_strided_rows(V, pad, dtype):
    t = make(7, V, 16, dtype, tail=True, pad=pad)
    wide = torch.full((7, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:20] = t["ids"]
    t["ids"] = wide[:, 4:20]
    a = check(t)  # the gradient's rows lie closer together than the logits'
    out = torch.full((7, V + pad), 9.0, dtype=DT[dtype], device="cuda")
    b = check(t, dlogits=out[:, :V])  # the same distances
    assert torch.equal(a["dz"], b["dz"]) and bool((out[:, V:] == 9.0).all())


@pytest.mark.parametrize("shift", [1, 3, 7])
def test_misaligned_start(shift):
    t = make(3, 2500, 16, "bf16", tail=True)
    buf = torch.zeros(3 * 2500 + 8, dtype=torch.bfloat16, device="cuda")
    odd = buf[shift:shift + 7500].view(3, 2500)
    odd.copy_(t["z"])
    t["z"] = odd
    check(t)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [600, 40001])
def test_in_place(V, tail):
    t = make(9, V, 30, "bf16", tail=tail)
    want = check(t)
    z = t["z"].clone()
    loss, rows = dgr.topk_distill(z, t["ids"], t["t"], tau=t["tau"], teacher_lse=t["lse"], weights=t["w"], scale=t["scale"],
                                  dlogits=z)
    assert torch.equal(z, want["dz"]) and torch.equal(rows, want["rows"]) and torch.equal(loss, want["loss"])


def test_dloss():
    t = make(5, 1000, 16, "fp32")
    up = torch.tensor([-2.0], device="cuda")
    same = dict(tau=t["tau"], weights=t["w"], scale=t["scale"])
    a = dgr.topk_distill_backward(t["z"], t["ids"], t["t"], **same)
    b = dgr.topk_distill_backward(t["z"], t["ids"], t["t"], dloss=up, **same)
    assert torch.equal(-2.0 * a, b)


def test_no_rows():
    z = torch.zeros(0, 50, device="cuda")
    loss, rows = dgr.topk_distill(z, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), torch.zeros(0, 4, device="cuda"))
    assert float(loss) == 0.0 and rows.shape == (0,)
    assert dgr.topk_distill_backward(z, torch.zeros(0, 4, dtype=torch.int32, device="cuda"),
                                     torch.zeros(0, 4, device="cuda")).shape == (0, 50)


def test_canonical_lists_may_be_passed_as_they_are():
    t = make(30, 800, 32, "fp32", weights=False)
    ids, logits, probs = dgr.topk_canonicalize(t["ids"].contiguous(), t["t"])
    want = check(t)
    t["ids"], t["t"] = ids, logits
    got = check(t)
    assert torch.allclose(got["rows"], want["rows"], rtol=1e-5, atol=1e-6)


def test_rows_past_2_to_the_31_elements():
    T, V, ld = 3, 500, (1 << 30) + 3
    t = make(T, V, 8, "bf16", weights=False)
    wide = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((T, V), (ld, 1))
    wide.copy_(t["z"])
    t["z"] = wide
    check(t)
    check(t, dlogits=torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((T, V), (ld, 1)))


def test_many_rows():
    t = make(3000, 40, 4, "bf16", tail=True)
    check(t)


def _call(t):
    dz = torch.empty_like(t["z"])
    loss, rows = dgr.topk_distill(t["z"], t["ids"], t["t"], tau=t["tau"], teacher_lse=t["lse"], weights=t["w"],
                                  scale=t["scale"], dlogits=dz)
    return torch.cat([loss, rows, dz.float().reshape(-1)])


@pytest.mark.parametrize("T,V,dtype,tail", [(900, 1111, "bf16", True), (12, 65536, "bf16", False), (330, 20000, "fp32", True)])
def test_no_schedule_changes_a_bit(T, V, dtype, tail):
    t = make(T, V, 24, dtype, tail=tail)
    base = bits(_call(t))
    for sch in SCHEDULES:
        with schedule(*sch):
            assert (bits(_call(t)) == base).all(), sch
    assert (assert_replays_identical(lambda: _call(t), n=6) == base).all()


def test_another_stream_and_a_captured_graph():
    t = make(64, 4000, 16, "bf16", tail=True)
    want = _call(t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dz = torch.empty_like(t["z"])
    same = dict(tau=t["tau"], teacher_lse=t["lse"], weights=t["w"], scale=t["scale"])
    loss, rows = dgr.topk_distill(t["z"], t["ids"], t["t"], dlogits=dz, stream=side, **same)
    side.synchronize()
    assert torch.equal(torch.cat([loss, rows, dz.float().reshape(-1)]), want)
    ws = dgr.workspace(dgr.topk_distill_workspace_bytes(64))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dgr.topk_distill(t["z"], t["ids"], t["t"], dlogits=dz, loss=loss, row_loss=rows, ws=ws, **same)
    for _ in range(2):
        for v in (loss, rows, dz):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.cat([loss, rows, dz.float().reshape(-1)]), want)
