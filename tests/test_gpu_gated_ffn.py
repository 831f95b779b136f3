"""GPU results of the gated feed-forward and its gradient against the 64-bit form: sizes around the tiles,
experts without rows, strided rows, neighbours that hold NaN, far values, schedules, streams, graphs."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import more_operator_ref as ref
from gpu_util import assert_replays_identical
from test_gpu_schedule import SCHEDULES, schedule

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def make(counts, H, F, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + 7 * H + F)
    T, E = sum(counts), len(counts)

    def rows(n, scale=1.0):  # in rows of a larger buffer, whose other columns hold NaN
        buf = torch.full((T, n + pad), float("nan"), dtype=BF)
        buf[:, :n] = (scale * torch.randn(T, n, generator=g)).to(BF)
        return buf.cuda()[:, :n]

    w = lambda: (H ** -0.5 * torch.randn(E, F, H, generator=g)).to(BF).cuda()  # noqa: E731
    offs = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0)
    return dict(x=rows(H), w_gate=w(), w_up=w(), offs=offs.cuda(), cuts=offs.tolist(), gate=rows(F), up=rows(F, 0.7), dh=rows(F, 0.1))


def near(got, want, bound, what):
    err = (ref.d(got) - want).abs()
    assert (err <= bound).all(), (what, float((err / bound).max()))


def check_forward(t, act, **out):
    h = dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], act=act, **out)
    args = ref.d(t["x"]), ref.d(t["w_gate"]), ref.d(t["w_up"]), t["cuts"], act
    want, bounds = ref.ffn(*args), ref.ffn_bounds(*args)
    near(h, want[0], bounds[0], "h")
    for k, i in (("gate", 1), ("up", 2)):
        if k in out:
            near(out[k], want[i], bounds[i], k)
    return h


def check_backward(t, act, **more):
    got = dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"], act=act, **more)
    args = ref.d(t["dh"]), ref.d(t["gate"]), ref.d(t["up"]), act
    want, bounds = ref.pre_grads(*args), ref.pre_grad_bounds(*args)
    near(got["dgate"], want[0], bounds[0], "dgate")
    near(got["dup"], want[1], bounds[1], "dup")
    args = ref.d(got["dgate"]), ref.d(got["dup"]), ref.d(t["w_gate"]), ref.d(t["w_up"]), t["cuts"]
    near(got["dx"], ref.dx(*args), ref.dx_bound(*args), "dx")
    return got


SIZES = [([1], 8, 8), ([5], 64, 40), ([1, 0, 2], 72, 136), ([128, 129, 0, 3], 200, 264), ([0, 0, 300], 1000, 128),
         ([40, 41, 42, 43, 0, 1], 328, 520), ([256, 257], 64, 1040), ([1000, 300], 136, 2056), ([2100], 72, 8), ([1800, 0, 1300], 1000, 136),
         ([5000, 0, 4400], 1544, 72), ([700], 2048, 256), ([0, 33], 264, 8), ([513, 1, 255], 136, 392)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,H,F", SIZES)
def test_forward(counts, H, F, act):
    t = make(counts, H, F)
    T = sum(counts)
    h = check_forward(t, act, gate=torch.empty(T, F, dtype=BF, device="cuda"), up=torch.empty(T, F, dtype=BF, device="cuda"))
    assert torch.equal(check_forward(t, act), h)  # with and without the products stored


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,H,F", SIZES)
def test_backward(counts, H, F, act):
    check_backward(make(counts, H, F), act)


@pytest.mark.parametrize("T,H,F", [(1, 4096, 1024), (3, 512, 8192), (17, 1024, 2048), (1, 8, 16384)])
def test_few_tokens_of_one_expert(T, H, F):
    t = make([T], H, F)
    h = check_forward(t, "silu")
    got = dgr.gated_ffn(t["x"], t["w_gate"][0], t["w_up"][0])
    assert torch.equal(got, h)  # weights [F, H], no offsets
    check_backward(t, "silu")


@pytest.mark.parametrize("counts,H", [([130, 7, 0, 64], 264), ([5430, 7, 0, 4564], 1544)])
def test_strided_rows_and_what_lies_around_the_outputs(counts, H):
    t = make(counts, H, 200, pad=24)
    T, F = sum(counts), 200
    outs = {k: torch.full((T + 3, n + 40), 7.0, dtype=BF, device="cuda") for k, n in (("h", F), ("gate", F), ("up", F), ("dx", H), ("dgate", F), ("dup", F))}
    view = {k: v[:T, :H if k == "dx" else F] for k, v in outs.items()}
    check_forward(t, "silu", **{k: view[k] for k in ("h", "gate", "up")})
    check_backward(t, "gelu", **{k: view[k] for k in ("dx", "dgate", "dup")})
    for k, v in outs.items():
        n = view[k].shape[1]
        assert (v[T:] == 7).all() and (v[:, n:] == 7).all(), k


@pytest.mark.parametrize("tail,H", [(90, 136), (9900, 1544)])
def test_neighbours_with_nan(tail, H):
    """A row of NaN, or an expert of NaN, stays with itself."""
    t = make([100, 60, tail], H, 264)
    clean = check_forward(t, "silu")
    back = check_backward(t, "silu")
    for k in ("x", "dh", "gate"):
        t[k][100:160] = float("nan")
        t[k][7] = float("nan")
    t["w_up"][1] = float("inf")
    h = dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"])
    got = dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"])
    keep = torch.ones(160 + tail, dtype=torch.bool, device="cuda")
    keep[100:160] = keep[7] = False
    assert torch.equal(h[keep], clean[keep]) and h[~keep].isnan().all()
    for k in back:
        assert torch.equal(got[k][keep], back[k][keep]), k
    assert got["dx"][~keep].isnan().all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_values(act):
    """Products far from zero: the activation is 0 or its argument, its gradient finite."""
    a = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 90, -90, 200, -200, 1e4, -1e4, 1e15, -1e15, 1e30, -1e30], device="cuda").to(BF)
    t = dict(make([16], 8, 8), gate=a[:, None].repeat(1, 8).contiguous())
    got = dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"], act=act)
    assert got["dgate"].isfinite().all()
    args = ref.d(t["dh"][:10]), ref.d(t["gate"][:10]), ref.d(t["up"][:10]), act
    for k, w, b in zip(("dgate", "dup"), ref.pre_grads(*args), ref.pre_grad_bounds(*args)):
        near(got[k][:10], w, b, k)
    dh = ref.d(t["dh"])
    assert torch.equal(ref.d(got["dgate"])[11::2], torch.zeros(3, 8, dtype=torch.float64))
    near(got["dgate"][10::2], (dh * ref.d(t["up"]))[10::2], 2.0 ** -8 * (dh * ref.d(t["up"])).abs()[10::2] * 1.001, "dgate")


@pytest.mark.parametrize("counts,H", [([90, 50], 128), ([9900, 50], 1544)])
def test_in_place_gradients(counts, H):
    t = make(counts, H, 264)
    want = check_backward(t, "silu")
    gate, up = t["gate"].clone(), t["up"].clone()
    got = dgr.gated_ffn_backward(t["dh"], gate, up, t["w_gate"], t["w_up"], offs=t["offs"], dgate=gate, dup=up)
    assert got["dgate"] is gate and all(torch.equal(got[k], want[k]) for k in want)


def test_weights_gradients():
    """Through the grouped weight gradient, added to what is there, with and without offsets."""
    counts, H, F = [300, 0, 77], 256, 128
    t = make(counts, H, F)
    old = torch.randn(3, F, H, device="cuda")
    dw = {"dw_gate": old.clone(), "dw_up": old.clone()}
    got = check_backward(t, "silu", x=t["x"], **dw)
    x, cuts = ref.d(t["x"]), t["cuts"]
    for k, g in (("dw_gate", "dgate"), ("dw_up", "dup")):
        g = ref.d(got[g])
        for e in range(3):
            rows = slice(cuts[e], cuts[e + 1])
            want = ref.d(old[e]) + g[rows].t() @ x[rows]
            bound = (1.2 * counts[e] + 20) * ref.U * (g[rows].abs().t() @ x[rows].abs()) + 2 * ref.U * (want.abs() + 1)
            near(dw[k][e], want, bound, k)
    one = make([40], H, F)
    a = torch.zeros(F, H, device="cuda")
    b = torch.zeros(1, F, H, device="cuda")
    dgr.gated_ffn_backward(one["dh"], one["gate"], one["up"], one["w_gate"][0], one["w_up"][0], x=one["x"], dw_gate=a)
    dgr.gated_ffn_backward(one["dh"], one["gate"], one["up"], one["w_gate"], one["w_up"], offs=one["offs"], x=one["x"], dw_gate=b)
    assert torch.equal(a, b[0]) and a.any()


@pytest.mark.parametrize("cuts", [[0, 10, 5, 20], [1, 5, 9, 20], [0, 5, 9, 19], [0, 5, 30, 20], [0, -4, 9, 20], [0, 1 << 40, 9, 20]])
def test_offsets_out_of_order(cuts):
    """Recorded in the status word; nothing is written."""
    t = make([5, 4, 11], 64, 72)
    ws = dgr.workspace(dgr.gated_ffn_workspace_bytes(10000, 1544, 72, 3))
    out = {k: torch.full((20, 72), 3.0, dtype=BF, device="cuda") for k in ("h", "gate", "up")}
    offs = torch.tensor(cuts, dtype=torch.int64, device="cuda")
    dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=offs, ws=ws, **out)
    assert dgr.read_device_status(ws, clear=True) == 1
    assert all((v == 3).all() for v in out.values())
    dx = torch.full((20, 64), 3.0, dtype=BF, device="cuda")
    dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=offs, ws=ws, dx=dx)
    assert dgr.read_device_status(ws, clear=True) == 1 and (dx == 3).all()
    many = make([5, 4, 9991], 1544, 72)  # the form for many rows
    # 9980 rows more in the last expert; where the third offset lies beyond the end it goes along (0, 5, 30, 10000 are in order)
    moved = cuts[:2] + [cuts[2] + (9980 if cuts[2] > cuts[3] else 0), cuts[3] + 9980]
    offs = torch.tensor(moved, dtype=torch.int64, device="cuda")
    dx = torch.full((10000, 1544), 3.0, dtype=BF, device="cuda")
    dgr.gated_ffn_backward(many["dh"], many["gate"], many["up"], many["w_gate"], many["w_up"], offs=offs, ws=ws, dx=dx)
    assert dgr.read_device_status(ws, clear=True) == 1 and (dx == 3).all()
    h = dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], ws=ws)  # the workspace goes on
    assert dgr.read_device_status(ws) == 0 and torch.equal(h, check_forward(t, "silu"))


def test_no_rows():
    t = make([0, 0], 64, 72)
    assert dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"]).shape == (0, 72)
    assert dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"])["dx"].shape == (0, 64)


def test_rows_do_not_depend_on_their_company():
    """The same row alone, in a batch, and behind other experts' rows has the same bits."""
    t = make([260, 140], 520, 392)
    h = check_forward(t, "silu")
    dx = check_backward(t, "silu")["dx"]
    for r, e in ((0, 0), (131, 0), (259, 0), (260, 1), (399, 1)):
        assert torch.equal(dgr.gated_ffn(t["x"][r:r + 1], t["w_gate"][e], t["w_up"][e])[0], h[r])
        one = [t[k][r:r + 1] for k in ("dh", "gate", "up")]
        assert torch.equal(dgr.gated_ffn_backward(*one, t["w_gate"][e], t["w_up"][e])["dx"][0], dx[r])


@pytest.mark.parametrize("counts,H,F", [([300, 1, 500, 0, 224], 264, 520), ([2, 0, 3], 512, 2048), ([5500, 4500], 1544, 264)])
def test_schedules_streams_and_replays(counts, H, F):
    t = make(counts, H, F)

    def run():
        h = dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"])
        b = dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"])
        return torch.cat([h.reshape(-1), b["dx"].reshape(-1), b["dgate"].reshape(-1)]).float()

    want = run()
    for s in SCHEDULES:
        with schedule(*s):
            assert torch.equal(run(), want), s
    assert_replays_identical(run, n=6)
    side = torch.cuda.Stream()
    h = dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], stream=side)
    side.synchronize()
    assert torch.equal(h, check_forward(t, "silu"))


def test_two_graphs_that_share_a_workspace():
    """Captured calls of other sizes, replayed in turn with new inputs."""
    ws = dgr.workspace(dgr.gated_ffn_workspace_bytes(10500, 1544, 72, 2))
    cases = []
    for counts, H, F in (([200, 60], 136, 264), ([3], 512, 1024), ([5700, 4800], 1544, 72)):
        t = make(counts, H, F)
        out = {"h": torch.empty(sum(counts), F, dtype=BF, device="cuda")}
        back = {k: torch.empty(sum(counts), n, dtype=BF, device="cuda") for k, n in (("dx", H), ("dgate", F), ("dup", F))}

        def call(t=t, out=out, back=back):
            dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], ws=ws, **out)
            dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"], ws=ws, **back)

        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        cases.append((g, t, out, back, call))
    for _ in range(2):
        for g, t, out, back, call in cases:
            t["x"].copy_(torch.randn_like(t["x"]))
            t["dh"].copy_(torch.randn_like(t["dh"]))
            g.replay()
            got = [v.clone() for v in (*out.values(), *back.values())]
            call()
            assert all(torch.equal(a, b) for a, b in zip(got, (*out.values(), *back.values())))
    assert dgr.read_device_status(ws) == 0
