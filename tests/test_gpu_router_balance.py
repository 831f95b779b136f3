"""GPU results of the router balance loss, its counts and its gradient against the 64-bit form.

Expert counts that take each layout of a row (one to thirty-two lanes, vectors and single elements),
packed groups with empty and fully masked ones, masked tokens that hold NaN, -inf logits, ids left
out, strided and misaligned rows, no tokens, launch schedules, replays, other streams.
"""
import numpy as np
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import operator_ref as ref
from gpu_util import assert_replays_identical, bits
from test_gpu_schedule import SCHEDULES, schedule

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
COEFF = 0.37


def make(N, E, K, dtype, offs=None, masked=False, pad=0, spread=1.5, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * N + E)
    buf = torch.full((N, E + pad), float("nan"), dtype=DT[dtype])
    buf[:, :E] = (spread * torch.randn(N, E, generator=g)).to(DT[dtype])
    ids = torch.randint(-1, E, (N, K), generator=g, dtype=torch.int32)
    mask = (torch.rand(N, generator=g) > 0.3) if masked else None
    x = buf.cuda()[:, :E]
    return dict(x=x, ids=ids.cuda(), mask=None if mask is None else mask.cuda(),
                offs=None if offs is None else torch.tensor(offs, dtype=torch.int64, device="cuda"))


def check(t, score, dloss=None, grad_into=None, accumulate=False):
    x, ids, mask, offs = t["x"], t["ids"], t["mask"], t["offs"]
    N, E = x.shape
    loss, counts, tokens = dgr.router_balance(x, ids, COEFF, offs=offs, mask=mask, score=score)
    up = None if dloss is None else torch.tensor([dloss], device="cuda")
    before = None if not accumulate else ref.d(grad_into)
    got = dgr.router_balance_backward(x, counts, tokens, ids.shape[1], COEFF, offs=offs, mask=mask, score=score,
                                      dloss=up, dlogits=grad_into, accumulate=accumulate)
    cpu_mask = None if mask is None else mask.cpu()
    v = ref.d(x)
    if cpu_mask is not None:
        v[cpu_mask == 0] = 0.0  # whatever a masked token holds
    v.requires_grad_()
    wl, wc, wt = ref.balance(v, ids.cpu(), COEFF, None if offs is None else offs.tolist(), cpu_mask, score)
    assert torch.equal(counts.cpu().long(), wc) and torch.equal(tokens.cpu().long(), wt)
    # a probability: an exponential of an exponent up to R (a rounding of R), a sum of E, a quotient;
    # its sum over tokens: a lane's rows, lanes, warps, tiles; the dot with the counts
    R = ref.finite_range(v.detach()) if N else 0.0
    rel = (64 + 4 * R + 2 * (N // 256 + 8) + E // 32) * ref.U
    assert abs(float(loss) - float(wl)) <= rel * float(wl) + 1e-40, (float(loss), float(wl))
    if wl.requires_grad:
        want = torch.autograd.grad(wl, v)[0] * (1.0 if dloss is None else float(up))
    else:
        want = torch.zeros_like(v)
    want = torch.where(torch.isfinite(v.detach()), want, torch.zeros_like(want))
    # terms: a p c and a p (c . p)
    bound = torch.zeros_like(want)
    p = ref.balance_scores(v.detach(), score)
    cuts = [0, N] if offs is None else offs.tolist()
    for s in range(len(cuts) - 1):
        rows = slice(cuts[s], cuts[s + 1])
        if int(wt[s]):
            a = abs(COEFF * (1.0 if dloss is None else dloss)) * E / ((len(cuts) - 1) * ids.shape[1] * int(wt[s]) ** 2)
            c = wc[s].double()
            bound[rows] = a * rel * p[rows] * (c + (p[rows] * c).sum(1, keepdim=True))
    if accumulate:
        live = torch.ones(N, dtype=torch.bool) if cpu_mask is None else cpu_mask != 0
        want = torch.where(live[:, None], want, torch.zeros_like(want)) + before
    bound = bound + ref.half_ulp(x.dtype) * want.abs() + 1e-40
    err = (ref.d(got) - want).abs()
    assert (err <= bound).all(), float((err / bound).max())
    return loss, counts, tokens, got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,E,K", [(1, 1, 1), (1, 8, 2), (5, 3, 3), (257, 8, 2), (100, 16, 4), (77, 33, 1), (130, 60, 6),
                                   (64, 64, 8), (300, 128, 8), (61, 130, 2), (45, 256, 4), (33, 300, 3), (20, 512, 8),
                                   (18, 1000, 5), (9, 1023, 2), (12, 1024, 16)])
def test_sizes(N, E, K, dtype, score):
    check(make(N, E, K, dtype), score, dloss=1.7)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tiles(score):
    check(make(3001, 128, 8, "fp32", masked=True), score)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [8, 60, 129])
def test_groups(E, dtype):
    N = 700
    t = make(N, E, 2, dtype, offs=[0, 0, 1, 1, 200, 457, 457, 600, N, N], masked=True)
    t["mask"][457:600] = False  # a group with tokens, none of them valid
    x = t["x"].clone()
    x[~t["mask"]] = float("nan")
    t["x"] = x
    loss, counts, tokens, grad = check(t, "softmax", dloss=0.3)
    assert int(tokens[6]) == 0 and not bool(counts[6].any())
    assert not bool(grad[~t["mask"]].any())


def test_one_group_by_offsets_is_the_group_without():
    t = make(500, 32, 4, "bf16")
    a = check(t, "softmax")
    t["offs"] = torch.tensor([0, 500], dtype=torch.int64, device="cuda")
    b = check(t, "softmax")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_many_groups():
    cuts = sorted([0, 3000] + np.random.RandomState(3).randint(0, 3001, 1023).tolist())
    check(make(3000, 16, 2, "fp32", offs=cuts), "softmax")


def test_largest_sizes_together():
    cuts = sorted([0, 2000] + np.random.RandomState(4).randint(0, 2001, 1023).tolist())
    check(make(2000, 1024, 2, "bf16", offs=cuts), "softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinities(score):
    t = make(40, 24, 2, "fp32")
    t["x"][3] = float("-inf")          # a row that leaves nothing
    t["x"][5, :20] = float("-inf")     # experts closed to a token
    t["x"][6, :23] = float("-inf")
    t["x"][7] = -3.0e38                # the type's lowest values
    t["x"][8] = -200.0                 # far below 0: the sigmoids underflow, their shares do not
    t["x"][8, 4] = -199.0
    _, _, _, grad = check(t, score)
    assert not bool(grad[3].any()) and not bool(grad[5, :20].any())
    assert bool(torch.isfinite(grad).all())


def test_ids_left_out_are_recorded():
    t = make(200, 16, 4, "fp32")
    want = dgr.router_balance(t["x"], t["ids"], COEFF)
    ws = dgr.workspace(dgr.router_balance_workspace_bytes(200, 16))
    got = dgr.router_balance(t["x"], torch.where(t["ids"] < 0, 99, t["ids"]), COEFF, ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert dgr.read_device_status(ws, clear=True) == 1
    got = dgr.router_balance(t["x"], t["ids"], COEFF, ws=ws)  # the workspace serves on
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and dgr.read_device_status(ws) == 0


@pytest.mark.parametrize("offs", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99], [0, -5, 60, 100], [0, 50, 200, 100]])
def test_offsets_outside_their_contract(offs):
    t = make(100, 16, 2, "fp32", offs=offs)
    ws = dgr.workspace(dgr.router_balance_workspace_bytes(100, 16, 3))
    loss = torch.full((1,), 7.0, device="cuda")
    counts = torch.full((3, 16), 5, dtype=torch.int32, device="cuda")
    tokens = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    dgr.router_balance(t["x"], t["ids"], COEFF, offs=t["offs"], loss=loss, counts=counts, tokens=tokens, ws=ws)
    assert dgr.read_device_status(ws) == 1
    assert float(loss) == 7.0 and bool((counts == 5).all()) and bool((tokens == 5).all())
    assert bool(torch.isfinite(dgr.router_balance_backward(t["x"], counts, tokens, 2, COEFF, offs=t["offs"])).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,pad", [(64, 4), (64, 1), (60, 4), (7, 9)])
def test_strided_rows(E, pad, dtype):
    t = make(90, E, 2, dtype, pad=pad)
    wide_ids = torch.full((90, 5), 99, dtype=torch.int32, device="cuda")
    wide_ids[:, 1:3] = t["ids"]
    t["ids"] = wide_ids[:, 1:3]
    check(t, "softmax")


def test_misaligned_start():
    t = make(50, 64, 2, "bf16")
    buf = torch.zeros(50 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(50, 64)
    odd.copy_(t["x"])
    t["x"] = odd
    check(t, "softmax")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_accumulate(dtype):
    t = make(150, 40, 2, dtype, masked=True)
    first = torch.randn(150, 40, generator=torch.Generator().manual_seed(5)).mul(1e-3).to(DT[dtype]).cuda()
    check(t, "softmax", grad_into=first.clone(), accumulate=True)


def test_no_tokens():
    x = torch.zeros(0, 8, device="cuda")
    loss, counts, tokens = dgr.router_balance(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), COEFF)
    assert float(loss) == 0.0 and not bool(counts.any()) and int(tokens) == 0
    assert dgr.router_balance_backward(x, counts, tokens, 2, COEFF).shape == (0, 8)
    t = make(50, 8, 2, "fp32")
    t["mask"] = torch.zeros(50, dtype=torch.uint8, device="cuda")
    loss, counts, tokens, grad = check(t, "softmax")
    assert float(loss) == 0.0 and int(tokens) == 0 and not bool(grad.any())


def test_rows_past_2_to_the_31_elements():
    N, E, ld = 3, 40, (1 << 30) + 4
    t = make(N, E, 2, "bf16")
    wide = torch.empty((N - 1) * ld + E, dtype=torch.bfloat16, device="cuda").as_strided((N, E), (ld, 1))
    wide.copy_(t["x"])
    t["x"] = wide
    check(t, "softmax")


def _call(t, score="softmax"):
    loss, counts, tokens = dgr.router_balance(t["x"], t["ids"], COEFF, offs=t["offs"], mask=t["mask"], score=score)
    g = dgr.router_balance_backward(t["x"], counts, tokens, t["ids"].shape[1], COEFF, offs=t["offs"], mask=t["mask"],
                                    score=score)
    return torch.cat([loss, counts.reshape(-1).float(), tokens.float(), g.float().reshape(-1)])


@pytest.mark.parametrize("N,E,dtype,offs", [(20000, 64, "fp32", None), (9000, 128, "bf16", [0, 10, 10, 4000, 9000])])
def test_no_schedule_changes_a_bit(N, E, dtype, offs):
    t = make(N, E, 4, dtype, offs=offs, masked=True)
    base = bits(_call(t))
    for sch in SCHEDULES:
        with schedule(*sch):
            assert (bits(_call(t)) == base).all(), sch
    assert (assert_replays_identical(lambda: _call(t), n=6) == base).all()


def test_another_stream_and_a_captured_graph():
    t = make(5000, 64, 4, "fp32")
    want = _call(t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    loss, counts, tokens = dgr.router_balance(t["x"], t["ids"], COEFF, stream=side)
    g = dgr.router_balance_backward(t["x"], counts, tokens, 4, COEFF, stream=side)
    side.synchronize()
    assert torch.equal(torch.cat([loss, counts.reshape(-1).float(), tokens.float(), g.reshape(-1)]), want)
    ws = dgr.workspace(dgr.router_balance_workspace_bytes(5000, 64))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dgr.router_balance(t["x"], t["ids"], COEFF, loss=loss, counts=counts, tokens=tokens, ws=ws)
        dgr.router_balance_backward(t["x"], counts, tokens, 4, COEFF, dlogits=g)
    for _ in range(2):  # the workspace is ready again after each replay
        for v in (loss, counts, tokens, g):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(torch.cat([loss, counts.reshape(-1).float(), tokens.float(), g.reshape(-1)]), want)
