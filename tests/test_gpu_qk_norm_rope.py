"""GPU results of the norm and rotation of queries and keys, and their gradients, against the 64-bit form:
head sizes that take each layout of a head, partial rotations, packed, transposed and misaligned heads,
zeros and far positions, positions outside the table, schedules, streams, graphs."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import more_operator_ref as ref
from gpu_util import assert_replays_identical
from test_gpu_schedule import SCHEDULES, schedule

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def table(P, R, base=10000.0):
    freq = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    ang = torch.arange(P, dtype=torch.float64)[:, None] * freq
    return torch.cos(ang).float().cuda(), torch.sin(ang).float().cuda()


def make(T, A, B, D, R, dtype, seed=0, packed=False, w="same", P=5000):
    g = torch.Generator().manual_seed(seed + 100 * D + T)
    dt = DT[dtype]
    r = lambda *s: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
    if packed:
        row = r(T, (A + 2 * B) * D + 2)
        q, k = row[:, :A * D].view(T, A, D), row[:, A * D:(A + B) * D].view(T, B, D)
    else:
        q, k = r(T, A, D), r(T, B, D)
    wdt = {"same": dt, "fp32": torch.float32, "none": None}[w]
    weight = lambda: None if wdt is None else (1 + 0.3 * torch.randn(D, generator=g)).to(wdt).cuda()  # noqa: E731
    c, s = table(P, R)
    return dict(q=q if A else None, k=k if B else None, cos=c, sin=s, positions=torch.randint(0, P, (T,), generator=g, dtype=torch.int32).cuda(),
                w_q=weight() if A else None, w_k=weight() if B else None), (r(T, A, D) if A else None, r(T, B, D) if B else None)


def near(got, want, bound, what):
    assert got.shape == want.shape
    err = (ref.d(got) - want).abs()
    assert (err <= bound).all(), (what, float((err / bound).max()))


def angles(t):
    at = t["positions"].long()
    return ref.d(t["cos"][at]), ref.d(t["sin"][at])


def check_forward(t, inter, **out):
    got = dgr.qk_norm_rope(**t, eps=EPS, interleaved=inter, **out)
    c, s = angles(t)
    for name, y in zip("qk", got):
        if t[name] is None:
            assert y is None
            continue
        args = ref.d(t[name]), ref.d(t["w_" + name]), c, s, EPS, inter
        near(y, ref.qk(*args), ref.qk_bound(*args, t[name].dtype), name)
    return got


def check_backward(t, dy, inter, **more):
    got = dgr.qk_norm_rope_backward(*dy, **t, eps=EPS, interleaved=inter, **more)
    c, s = angles(t)
    for name, g in zip("qk", dy):
        if g is None:
            continue
        args = ref.d(g), ref.d(t[name]), ref.d(t["w_" + name]), c, s, EPS, inter
        (dv, dw), (bv, bw) = ref.qk_grads(*args), ref.qk_grad_bounds(*args, g.dtype)
        near(got["d" + name], dv, bv, "d" + name)
        if t["w_" + name] is not None:
            near(got["dw_" + name], dw, bw, "dw_" + name)
    return got


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,A,B,D,R", [(1, 1, 1, 2, 2), (3, 4, 1, 64, 64), (17, 3, 2, 128, 128), (9, 8, 2, 128, 64), (5, 2, 2, 80, 40),
                                       (33, 5, 1, 96, 32), (4, 6, 3, 42, 20), (7, 2, 1, 18, 18), (6, 2, 2, 512, 512), (11, 3, 1, 256, 2),
                                       (3, 2, 1, 510, 254), (129, 32, 8, 128, 128), (2, 40, 0, 64, 64), (5, 0, 3, 32, 16), (300, 1, 1, 20, 8)])
def test_sizes(T, A, B, D, R, dtype, inter):
    t, dy = make(T, A, B, D, R, dtype)
    check_forward(t, inter)
    check_backward(t, dy, inter)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("w", ["fp32", "none"])
def test_weights_of_other_types(w, dtype):
    t, dy = make(20, 4, 2, 64, 64, dtype, w=w)
    check_forward(t, False)
    got = check_backward(t, dy, False)
    assert ("dw_q" in got) == (w != "none")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_packed_rows_and_in_place(dtype):
    """q and k cut out of one row that starts at no multiple of 16 bytes; outputs over the inputs."""
    t, dy = make(21, 6, 2, 64, 32, dtype, packed=True)
    want = check_forward(t, False)
    back = check_backward(t, dy, False)
    rest = t["q"]._base[:, 8 * 64:].clone()
    got = dgr.qk_norm_rope(**t, eps=EPS, q_out=t["q"], k_out=t["k"])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(t["q"]._base[:, 8 * 64:], rest)
    t, dy = make(21, 6, 2, 64, 32, dtype, packed=True)
    got = dgr.qk_norm_rope_backward(*dy, **t, eps=EPS, dq=dy[0], dk=dy[1])
    assert all(torch.equal(got[k], back[k]) for k in back)
    # gradients into one packed row's places
    row = torch.full((21, 10 * 64), 5.0, dtype=DT[dtype], device="cuda")
    t, dy = make(21, 6, 2, 64, 32, dtype, packed=True)
    got = dgr.qk_norm_rope_backward(*dy, **t, eps=EPS, dq=row[:, :384].view(21, 6, 64), dk=row[:, 384:512].view(21, 2, 64))
    assert all(torch.equal(got[k], back[k]) for k in back) and (row[:, 512:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_heads_before_tokens(dtype):
    t, dy = make(19, 4, 2, 96, 96, dtype)
    want = check_forward(t, True)
    t["q"] = t["q"].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(4, 19, 96, dtype=DT[dtype], device="cuda").transpose(0, 1)
    got = check_forward(t, True, q_out=out)
    assert got[0] is out and torch.equal(got[0], want[0])
    check_backward(t, dy, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_far_positions_zeros_and_large_values(dtype):
    t, dy = make(6, 2, 2, 64, 64, dtype, P=200000)
    t["positions"][:] = torch.tensor([0, 199999, 199998, 131072, 1, 0])
    t["q"][2] = 0  # r = eps^(-1/2)
    t["k"][3] = 1e15
    t["k"][4] *= 1e-12
    check_forward(t, False)
    check_backward(t, dy, False)


def test_nan_stays_in_its_head():
    t, dy = make(8, 4, 2, 64, 64, "bf16")
    want = dgr.qk_norm_rope(**t)
    back = dgr.qk_norm_rope_backward(*dy, **t)
    t["q"][3, 1, 5] = float("nan")
    got = dgr.qk_norm_rope(**t)
    assert got[0][3, 1].isnan().all() and torch.equal(got[1], want[1])
    keep = torch.ones(8, 4, dtype=torch.bool, device="cuda")
    keep[3, 1] = False
    assert torch.equal(got[0][keep], want[0][keep])
    again = dgr.qk_norm_rope_backward(*dy, **t)
    assert torch.equal(again["dq"][keep], back["dq"][keep]) and torch.equal(again["dw_k"], back["dw_k"]) and again["dw_q"].isnan().all()


@pytest.mark.parametrize("bad", [-1, 5000, 2 ** 31 - 1, -2 ** 31])
def test_positions_outside_the_table(bad):
    t, dy = make(9, 4, 2, 64, 64, "fp32")
    t["positions"][4] = bad
    ws = dgr.workspace(dgr.qk_norm_rope_workspace_bytes(9, 4, 2, 64))
    q, k = dgr.qk_norm_rope(**t, ws=ws)
    assert dgr.read_device_status(ws, clear=True) == 1 and not q[4].any() and not k[4].any()
    got = dgr.qk_norm_rope_backward(*dy, **t, ws=ws)
    assert dgr.read_device_status(ws, clear=True) == 1 and not got["dq"][4].any() and not got["dk"][4].any()
    # as without that token
    keep = torch.arange(9, device="cuda") != 4
    u = {n: v[keep].contiguous() if n in ("q", "k", "positions") else v for n, v in t.items()}
    c, s = angles(u)
    args = ref.d(dy[0][keep]), ref.d(u["q"]), ref.d(u["w_q"]), c, s, 1e-6, False
    near(got["dw_q"], ref.qk_grads(*args)[1], ref.qk_grad_bounds(*args, torch.float32)[1], "dw_q")
    assert torch.equal(q[keep], dgr.qk_norm_rope(**u)[0])


def test_accumulate_and_no_tokens():
    t, dy = make(50, 4, 2, 64, 64, "fp32")
    got = check_backward(t, dy, False)
    old = {"dw_q": torch.randn(64, device="cuda"), "dw_k": torch.randn(64, device="cuda")}
    new = {k: v.clone() for k, v in old.items()}
    dgr.qk_norm_rope_backward(*dy, **t, eps=EPS, accumulate=True, **new)
    assert all(torch.equal(new[k], old[k] + got[k]) for k in old)
    t, dy = make(0, 4, 2, 64, 64, "fp32")
    assert dgr.qk_norm_rope(**t)[0].shape == (0, 4, 64)
    got = dgr.qk_norm_rope_backward(*dy, **t)
    assert not got["dw_q"].any() and not got["dw_k"].any()
    kept = {k: v.clone() for k, v in old.items()}
    dgr.qk_norm_rope_backward(*dy, **t, accumulate=True, **kept)
    assert all(torch.equal(kept[k], old[k]) for k in old)


def test_many_tokens_in_one_workspace_after_few():
    ws = dgr.workspace(dgr.qk_norm_rope_workspace_bytes(6000, 4, 1, 64))
    for T in (6000, 3, 700):
        t, dy = make(T, 4, 1, 64, 64, "bf16")
        check_backward(t, dy, False, ws=ws)


@pytest.mark.parametrize("T,A,B,D,R,dtype", [(700, 8, 2, 128, 128, "bf16"), (13, 3, 1, 42, 20, "fp32"), (1, 32, 8, 128, 128, "bf16")])
def test_schedules_streams_and_replays(T, A, B, D, R, dtype):
    t, dy = make(T, A, B, D, R, dtype)

    def run(stream=None):
        y = dgr.qk_norm_rope(**t, stream=stream)
        g = dgr.qk_norm_rope_backward(*dy, **t, stream=stream)
        if stream is not None:
            stream.synchronize()
        return torch.cat([v.reshape(-1).float() for v in (*y, *g.values())])

    want = run()
    for s in SCHEDULES:
        with schedule(*s):
            assert torch.equal(run(), want), s
    assert_replays_identical(run, n=6)
    torch.cuda.synchronize()
    assert torch.equal(run(torch.cuda.Stream()), want)


def test_captured():
    t, dy = make(60, 4, 2, 64, 64, "bf16")
    ws = dgr.workspace(dgr.qk_norm_rope_workspace_bytes(60, 4, 2, 64))
    out = {"q_out": torch.empty_like(t["q"]), "k_out": torch.empty_like(t["k"])}
    back = {"dq": torch.empty_like(t["q"]), "dk": torch.empty_like(t["k"]), "dw_q": torch.empty(64, device="cuda"), "dw_k": torch.empty(64, device="cuda")}

    def call():
        dgr.qk_norm_rope(**t, ws=ws, **out)
        dgr.qk_norm_rope_backward(*dy, **t, ws=ws, **back)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        t["q"].copy_(torch.randn_like(t["q"]))
        g.replay()
        got = [v.clone() for v in (*out.values(), *back.values())]
        call()
        assert all(torch.equal(a, b) for a, b in zip(got, (*out.values(), *back.values())))
