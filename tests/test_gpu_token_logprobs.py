"""GPU results of the token log probabilities, entropies, top alternatives and their gradient against the
64-bit form: rows of every length and alignment, rows left out, masks that leave one element or none,
logits far from zero, equal logits, lists longer than a row, schedules, streams, graphs."""
import math

import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import more_operator_ref as ref
from gpu_util import assert_replays_identical
from test_gpu_schedule import SCHEDULES, schedule

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
INF = math.inf


def make(T, V, dtype, seed=0, pad=0, lead=0, scale=3.0):
    """Rows of a larger buffer whose other columns hold NaN; the first starts `lead` elements into it."""
    g = torch.Generator().manual_seed(seed + V + T)
    buf = torch.full((T * (V + pad) + lead,), float("nan"), dtype=DT[dtype])
    rows = buf[lead:].view(T, V + pad)
    rows[:, :V] = (scale * torch.randn(T, V, generator=g)).to(DT[dtype])
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if T > 2:
        ids[T // 2] = -1
    return buf.cuda()[lead:].view(T, V + pad)[:, :V], ids.cuda()


def near(got, want, bound, what):
    got, top = ref.d(got), torch.finfo(got.dtype).max
    want = torch.where(want.abs() > top, want * INF, want)  # what the type cannot hold rounds to infinity
    same = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), same) and torch.equal(got[~same], want[~same]), what
    err = (got - want).abs()[same]
    assert (err <= bound[same]).all(), (what, float((err / bound[same]).max()))


def check_forward(z, ids, tau=1.0, top=0, **more):
    got = dgr.token_logprobs(z, ids, tau=tau, top=top, **more)
    T, V = z.shape
    v = ref.d(z)
    on = torch.ones(T, dtype=torch.bool) if ids is None else (ids.cpu() >= 0) & (ids.cpu() < V)
    lp, H, lse = ref.logp_rows(v, tau)
    at = torch.zeros(T, dtype=torch.long) if ids is None else torch.where(on, ids.cpu().long(), 0)
    lp_at = lp.gather(1, at[:, None])[:, 0]
    b_lp, b_H, b_lse = ref.logp_bounds(v, tau, lp_at)
    zero = lambda t: torch.where(on, t, 0.0)  # noqa: E731
    if ids is not None:
        near(got["logp"], zero(lp_at), zero(b_lp), "logp")
    near(got["entropy"], zero(H), zero(b_H), "entropy")
    near(got["lse"], zero(lse), zero(b_lse), "lse")
    m = v.amax(1)
    assert torch.equal(ref.d(got["stats"])[:, 0], zero(m))
    lns = torch.where(m == -INF, 0.0, ref.logp_rows(v - torch.where(m == -INF, 0.0, m)[:, None], tau)[2])
    lns = torch.where(m == -INF, 0.0, lns)
    near(got["stats"][:, 1], zero(lns), zero(b_lse), "ln s")
    if top:
        want, val = ref.top(v, top)
        want[~on], val[~on] = -1, -INF
        assert torch.equal(got["top_ids"].cpu(), want)
        assert torch.equal(ref.d(got["top_logits"]), val)
        some = val > -INF
        wlp = torch.where(some, torch.where(some, val, 0.0) / tau - torch.where(torch.isfinite(lse), lse, 0.0)[:, None], -INF)
        near(got["top_logp"], wlp, b_lse[:, None] + 8 * ref.U * torch.where(some, wlp.abs() + (val / tau).abs(), 0.0), "top_logp")
    return got


def check_backward(z, ids, got, tau=1.0, dlogits=None, seed=0, only=None):
    T, V = z.shape
    g = torch.Generator().manual_seed(seed)
    a, b = torch.randn(T, generator=g), torch.randn(T, generator=g)
    a, b = (None if only == "entropy" else a), (None if only == "logp" else b)
    v, cpu = ref.d(z), None if ids is None else ids.cpu()
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"] if b is not None else None, dlogp=cuda(a), dentropy=cuda(b), tau=tau,
                                     dlogits=dlogits)
    near(dz, ref.logp_grad(v, cpu, ref.d(a), ref.d(b), tau), ref.logp_grad_bound(v, cpu, ref.d(a), ref.d(b), tau, z.dtype), "dlogits")
    return dz


LENGTHS = [1, 2, 7, 8, 33, 100, 1000, 1023, 4097, 8191, 16384, 50001]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", LENGTHS)
def test_lengths(V, dtype):
    for T, tau in ((1, 1.0), (5, 0.7)):
        z, ids = make(T, V, dtype)
        got = check_forward(z, ids, tau)
        check_backward(z, ids, got, tau)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,lead", [(1, 0), (0, 1), (3, 5), (7, 3), (8, 0)])
def test_rows_that_start_anywhere(pad, lead, dtype):
    for V in (15, 999, 5003):
        z, ids = make(6, V, dtype, pad=pad, lead=lead)
        got = check_forward(z, ids, top=9)
        want = check_backward(z, ids, got)
        # gradients at another alignment than the logits, their surroundings left as they are
        buf = torch.full((6 * (V + 2) + 3,), 5.0, dtype=DT[dtype], device="cuda")
        out = buf[3:].view(6, V + 2)[:, :V]
        assert torch.equal(check_backward(z, ids, got, dlogits=out), want)
        assert (buf[:3] == 5).all() and (buf[3:].view(6, V + 2)[:, V:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 5, 8), (2, 300, 128), (4, 4096, 128), (3, 65536, 20), (1, 131072, 64), (700, 2000, 5),
                                   (2, 262144, 128), (5, 50001, 1), (200, 9001, 100), (1, 1 << 20, 33)])
def test_top(T, V, K, dtype):
    z, ids = make(T, V, dtype)
    check_forward(z, ids, 1.3, K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_logits(dtype):
    """Ties go to the lowest index: all equal, two values, -0 beside +0, the tie at the list's end."""
    V = 40000
    z = torch.zeros(6, V, dtype=DT[dtype], device="cuda")
    z[1, ::3] = 1.0
    z[2, 1::2] = -0.0
    z[3] = torch.randint(0, 3, (V,), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    z[4, 39000:] = 2.0
    z[4, 17] = 2.0
    z[5] = -7.0
    z[5, 39999] = -6.0
    ids = torch.arange(6, dtype=torch.int32, device="cuda")
    for K in (1, 7, 128):
        got = check_forward(z, ids, top=K)
    check_backward(z, ids, got)
    z, ids = make(4, 3000, dtype, scale=1.0)
    z.copy_((z * 4).round() / 4)  # few values
    check_forward(z, ids, top=120)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [50, 20000])
def test_masks(V, dtype):
    """-inf and the type's lowest value: some, all but one, all."""
    z, ids = make(9, V, dtype)
    low = torch.finfo(DT[dtype]).min
    z[0, ::2] = -INF
    z[1] = -INF
    z[1, V - 1] = 3.0
    z[2] = -INF
    z[3, ::3] = low
    z[5] = low
    z[6] = low
    z[6, 7] = -2.0
    z[7, 1:] = -INF
    z[8] = -INF
    ids[:] = torch.tensor([1, V - 1, 3, 4, -1, 2, 7, 5, 0])
    ids[0] = 0
    got = check_forward(z, ids, top=20)  # row 0's token is masked: -inf
    check_backward(z, ids, got)
    check_forward(z, None, top=20)
    check_backward(z, None, dgr.token_logprobs(z), only="entropy")
    # with the list's length beyond what is left
    got = dgr.token_logprobs(z, ids, top=3)
    assert got["top_ids"][1].tolist() == [V - 1, -1, -1] and got["top_logits"][1].tolist() == [3.0, -INF, -INF]
    # a lone element: ln s = ln 2^d - d ln 2, d the rounding of m k; 2^d is off by up to 2 units (its approximation),
    # its logarithm and the product by one each: 4 units of 2^-23, not 0
    assert abs(float(got["logp"][1])) <= 8 * ref.U and abs(float(got["entropy"][1])) <= 8 * ref.U and float(got["logp"][2]) == -INF


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("at", [3e3, -3e3, 1e6, -2e8, 1e20, -1e33, 1e38])
def test_far_from_zero(at, dtype):
    """Rows around a far value: differences that the type still holds count, the row's place does not."""
    V = 9000
    g = torch.Generator().manual_seed(5)
    step = abs(at) * 2.0 ** (-7 if dtype == "bf16" else -22)
    z = (at + step * torch.randint(-3, 1, (4, V), generator=g)).to(DT[dtype]).cuda()
    z[1, ::2] = -INF
    z[2, 100:] = 0.0 if at < 0 else -1.0
    ids = torch.tensor([5, 1, 7, -1], dtype=torch.int32, device="cuda")
    for tau in (1.0, 1e-3, 1e4):
        got = dgr.token_logprobs(z, ids, tau=tau, top=3)
        v = ref.d(z)
        m = v.amax(1, keepdim=True)
        # the logits' distance to the maximum first: exact in both
        lp, H, lse = ref.logp_rows(v - m, tau)
        on = ids.cpu() >= 0
        lp_at = lp.gather(1, ids.cpu().long().clamp(min=0)[:, None])[:, 0]
        b_lp, b_H, b_lse = ref.logp_bounds(v - m, tau, lp_at)
        near(got["logp"], torch.where(on, lp_at, 0.0), b_lp, "logp")
        near(got["entropy"], torch.where(on, H, 0.0), b_H, "entropy")
        near(got["stats"][:, 1], torch.where(on, lse, 0.0), b_lse, "ln s")
        want, val = ref.top(v, 3)
        assert torch.equal(got["top_ids"].cpu()[on], want[on]) and torch.equal(ref.d(got["top_logits"])[on], val[on])
        a, b = torch.ones(4), torch.ones(4)
        dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=a.cuda(), dentropy=b.cuda(), tau=tau)
        near(dz, ref.logp_grad(v - m, ids.cpu(), ref.d(a), ref.d(b), tau), ref.logp_grad_bound(v - m, ids.cpu(), ref.d(a), ref.d(b), tau, z.dtype), "dz")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_nan_and_infinity(dtype):
    z, ids = make(6, 3000, dtype)
    clean = dgr.token_logprobs(z, ids, top=5)
    z[1, 2500], z[4, 7] = float("nan"), INF
    z[3] = float("nan")  # row 3 is left out
    got = dgr.token_logprobs(z, ids, top=5)
    for k in ("logp", "entropy", "lse"):
        assert got[k][[1, 4]].isnan().all() and torch.equal(got[k][[0, 2, 3, 5]], clean[k][[0, 2, 3, 5]]), k
    want, val = ref.top(ref.d(z), 5)
    assert torch.equal(got["top_ids"].cpu()[[1, 4]], want[[1, 4]]) and float(got["top_logits"][4, 0]) == INF
    dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=torch.ones(6, device="cuda"))
    assert dz[[1, 4]].isnan().all() and not dz[3].any() and dz[[0, 2, 5]].isfinite().all()


def test_rows_left_out_are_not_read_and_ids_out_of_range():
    z, ids = make(8, 500, "fp32")
    ids[:] = torch.tensor([3, -1, 499, 500, 2 ** 31 - 1, -2 ** 31, 0, 7])
    out = [1, 3, 4, 5]
    z[out] = float("nan")
    ws = dgr.workspace(256)
    got = dgr.token_logprobs(z, ids, top=4, ws=ws)
    assert dgr.read_device_status(ws, clear=True) == 1
    for k in ("logp", "entropy", "lse", "stats"):
        assert not got[k][out].any(), k
    assert (got["top_ids"][out] == -1).all() and (got["top_logp"][out] == -INF).all()
    dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=torch.ones(8, device="cuda"))
    assert not dz[out].any() and dz.isfinite().all()
    keep = [0, 2, 6, 7]
    check_forward(z[keep].contiguous(), ids[keep].contiguous(), top=4)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("only", ["logp", "entropy"])
def test_one_gradient_alone_and_in_place(only, dtype):
    z, ids = make(9, 7001, dtype, pad=3)
    got = check_forward(z, ids, 2.0)
    want = check_backward(z, ids, got, 2.0, only=only)
    assert torch.equal(_again(z, ids, got, only), want)


def _again(z, ids, got, only):
    g = torch.Generator().manual_seed(0)
    a, b = torch.randn(9, generator=g).cuda(), torch.randn(9, generator=g).cuda()
    out = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=a if only == "logp" else None,
                                      dentropy=b if only == "entropy" else None, tau=2.0, dlogits=z)
    assert out is z
    return out


def test_gradient_of_many_rows():
    z, ids = make(1500, 3001, "bf16")
    got = check_forward(z, ids, top=2)
    check_backward(z, ids, got)


def test_teacher_lists_for_the_distillation():
    """top_ids, top_logits and lse as topk_distill's ids, teacher and teacher_lse."""
    teacher, _ = make(12, 4001, "fp32", scale=2.0)
    student, _ = make(12, 4001, "fp32", seed=9)
    t = dgr.token_logprobs(teacher, tau=1.5, top=32)
    _, rows = dgr.topk_distill(student, t["top_ids"], t["top_logits"], tau=1.5, teacher_lse=t["lse"])
    v = ref.d(teacher)
    best = v.topk(32, dim=1)
    import operator_ref
    want = operator_ref.distill_rows(ref.d(student), best.indices, best.values, 1.5, torch.logsumexp(v / 1.5, 1))
    assert ((ref.d(rows) - want).abs() <= 1e-5 * want.abs() + 1e-5).all()


def test_no_rows():
    z, ids = make(0, 100, "bf16")
    got = dgr.token_logprobs(z, ids, top=3)
    assert got["logp"].shape == (0,) and got["top_ids"].shape == (0, 3)
    assert dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=got["logp"]).shape == (0, 100)


@pytest.mark.parametrize("T,V,K,dtype", [(400, 3000, 0, "bf16"), (3, 70000, 40, "fp32"), (60, 9001, 100, "bf16")])
def test_schedules_streams_and_replays(T, V, K, dtype):
    z, ids = make(T, V, dtype)
    one = torch.ones(T, device="cuda")

    def run(stream=None):
        got = dgr.token_logprobs(z, ids, top=K, stream=stream)
        dz = dgr.token_logprobs_backward(z, ids, got["stats"], got["entropy"], dlogp=one, dentropy=one, stream=stream)
        if stream is not None:
            stream.synchronize()
        return torch.cat([v.reshape(-1).float() for v in (*got.values(), dz)])

    want = run()
    for s in SCHEDULES:
        with schedule(*s):
            assert torch.equal(run(), want), s
    assert_replays_identical(run, n=6)
    torch.cuda.synchronize()
    assert torch.equal(run(torch.cuda.Stream()), want)


def test_captured_twice_with_one_workspace():
    ws = dgr.workspace(256)
    calls = []
    for T, V, K in ((30, 2000, 5), (2, 70000, 0)):
        z, ids = make(T, V, "bf16")
        out = {k: v for k, v in dgr.token_logprobs(z, ids, top=K, ws=ws).items()}
        dz, one = torch.empty_like(z), torch.ones(T, device="cuda")

        def call(z=z, ids=ids, K=K, out=out, dz=dz, one=one):
            dgr.token_logprobs(z, ids, top=K, ws=ws, **out)
            dgr.token_logprobs_backward(z, ids, out["stats"], out["entropy"], dlogp=one, dlogits=dz)

        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        calls.append((g, z, out, dz, call))
    for _ in range(3):
        for g, z, out, dz, call in calls:
            z.copy_(3 * torch.randn_like(z))
            g.replay()
            got = [v.clone() for v in (*out.values(), dz)]
            call()
            assert all(torch.equal(a, b) for a, b in zip(got, (*out.values(), dz)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,K,pad,lead", [(1, 1, 0, 0), (300, 1, 3, 1), (1000, 5, 0, 0), (4099, 60, 5, 3), (8150, 128, 2, 0), (16380, 20, 0, 0)])
def test_many_short_rows(V, K, pad, lead, dtype):
    """Rows beyond what the list warps of large CTAs hold at once: ties, masks, NaN, rows left out, far values among them."""
    T = 1300
    z, ids = make(T, V, dtype, pad=pad, lead=lead)
    z[::9] = 0.25
    z[1::9, ::2] = -INF
    z[2::9] = -INF
    z[3::9] = (z[3::9] * 2).round() / 2  # few values
    z[4::9, V // 2:] = torch.finfo(DT[dtype]).min
    z[5::9, : V // 3] = 40.0
    ids[6::9] = -1
    z[6::9] = float("nan")
    keep = torch.arange(T) % 9 != 6
    got = dgr.token_logprobs(z, ids, top=K, tau=1.3)
    some = check_forward(z[keep].contiguous(), ids[keep].contiguous(), 1.3, K)
    assert (got["top_ids"][~keep] == -1).all() and not got["logp"][~keep].any()
    for k in ("top_ids", "top_logits"):
        assert torch.equal(got[k][keep], some[k]), k
    assert_replays_identical(lambda: torch.cat([v.reshape(-1).float() for v in dgr.token_logprobs(z, ids, top=K, tau=1.3).values()]), n=3)
    # one far above the others, NaN in another row: neither reaches a third
    z, ids = make(T, max(V, 8), dtype)
    clean = dgr.token_logprobs(z, ids, top=1)
    z[5, 3], z[700, 7] = INF, float("nan")
    got = dgr.token_logprobs(z, ids, top=1)
    rest = [t for t in range(T) if t not in (5, 700)]
    assert all(torch.equal(got[k][rest], clean[k][rest]) for k in got) and int(got["top_ids"][5]) == 3
