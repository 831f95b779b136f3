"""GPU results of the block norms (forward and backward) against the 64-bit form.

Widths that take each layout of a row (a warp, a small and a large block, one element a load, the
widest rows), ragged and strided rows, every combination of norms and gates, one token and none,
in-place outputs, zero rows, rows past 2^31 elements, other streams, launch schedules and replays.
"""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import operator_ref as ref
from gpu_util import assert_replays_identical, bits
from test_gpu_schedule import SCHEDULES, schedule

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(T, H, dtype, gate="channel", post=True, pre=True, wdtype=None, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + H)
    dt, wdt = DT[dtype], DT[wdtype or dtype]

    def rows(scale):
        buf = torch.full((T, H + pad), float("nan"), dtype=dt)
        buf[:, :H] = (scale * torch.randn(T, H, generator=g)).to(dt)
        return buf.cuda()[:, :H]

    def w(*shape, mean=1.0):
        return (mean + 0.3 * torch.randn(*shape, generator=g)).to(wdt).cuda()

    t = dict(x=rows(2.0), y=rows(0.7), dh=rows(0.1), du=rows(0.1), w_post=w(H) if post else None,
             w_pre=w(H) if pre else None)
    t["gate"] = {"none": None, "channel": w(H, mean=0.5), "token": w(T, 1, mean=0.5)}[gate]
    return t


def check_forward(t, alpha=0.9, eps=1e-5, **kw):
    h, u = dgr.block_norm(t["x"], t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=alpha, w_pre=t["w_pre"],
                          eps=eps, **kw)
    args = [ref.d(t[k]) for k in ("x", "y", "w_post", "gate")] + [alpha, ref.d(t["w_pre"]), eps]
    wh, wu = ref.block_norm(*args)
    bh, bu = ref.block_norm_bounds(*args, t["x"].dtype)
    assert ((ref.d(h) - wh).abs() <= bh).all(), float(((ref.d(h) - wh).abs() - bh).max())
    if wu is None:
        assert u is None
    else:
        assert ((ref.d(u) - wu).abs() <= bu).all(), float(((ref.d(u) - wu).abs() - bu).max())
    return h, u


def check_backward(t, h, alpha=0.9, eps=1e-5, before=None, **kw):
    got = dgr.block_norm_backward(h, t["y"], t["dh"], t["du"], w_post=t["w_post"], gate=t["gate"], res_scale=alpha,
                                  w_pre=t["w_pre"], eps=eps, **kw)
    args = [ref.d(v) for v in (h, t["y"], t["dh"], t["du"], t["w_post"], t["gate"])] + [alpha, ref.d(t["w_pre"]), eps]
    want = ref.block_norm_grads(*args)
    bound = ref.block_norm_grad_bounds(*args)
    assert set(got) == set(bound)
    for k, v in got.items():
        w, b = want[k], bound[k]
        if before is not None and k in before:
            w = w + ref.d(before[k])
            b = b + ref.U * w.abs()
        b = b + ref.half_ulp(v.dtype) * w.abs() + 1e-40
        err = (ref.d(v) - w).abs()
        assert (err <= b).all(), (k, float((err / b).max()))
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (5, 7), (67, 64), (33, 100), (9, 256), (300, 264), (41, 512), (20, 513),
                                 (17, 1000), (19, 1024), (40, 1032), (700, 2048), (13, 2050), (9, 4096), (7, 5000),
                                 (5, 8192), (3, 12001), (4, 16384)])
def test_widths(T, H, dtype):
    t = make(T, H, dtype)
    h, _ = check_forward(t)
    check_backward(t, h)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "fp32"), ("fp32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_forms(dtype, wdtype, gate, post, pre):
    t = make(37, 136, dtype, gate, post, pre, wdtype)
    if not pre:
        t["du"] = None
    h, _ = check_forward(t, alpha=-0.4)
    check_backward(t, h, alpha=-0.4)


def test_norm_alone_and_without_dh():
    t = make(29, 320, "bf16", "none", False, True)
    t["y"] = None
    h, u = check_forward(t, alpha=1.0)
    assert h.data_ptr() == t["x"].data_ptr()
    got = check_backward(t, h, alpha=1.0)
    assert set(got) == {"dx", "dw_pre"}
    t["dh"] = None
    check_backward(t, h, alpha=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("H,pad", [(512, 8), (4096, 64), (1000, 3), (200, 1), (72, 4)])
def test_strided_rows(H, pad, dtype):
    t = make(21, H, dtype, "token", pad=pad)
    h, _ = check_forward(t)
    check_backward(t, h)


def test_misaligned_start():
    t = make(6, 64, "bf16")
    buf = torch.zeros(6 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(6, 64)
    odd.copy_(t["x"])
    t["x"] = odd
    h, _ = check_forward(t)
    check_backward(t, h)


def test_in_place():
    t = make(50, 768, "bf16")
    want_h, want_u = check_forward(t)
    x = t["x"].clone()
    h, u = dgr.block_norm(x, t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9, w_pre=t["w_pre"], eps=1e-5, h=x)
    assert h.data_ptr() == x.data_ptr() and torch.equal(h, want_h) and torch.equal(u, want_u)
    want = check_backward(t, want_h)
    dh = t["dh"].clone()
    got = dgr.block_norm_backward(want_h, t["y"], dh, t["du"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9,
                                  w_pre=t["w_pre"], eps=1e-5, dx=dh)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_accumulate():
    for gate in ("channel", "token"):
        t = make(45, 300, "fp32", gate)
        h, _ = check_forward(t)
        g = torch.Generator().manual_seed(9)
        first = {k: torch.randn(*s, generator=g).cuda() for k, s in
                 (("dw_post", (300,)), ("dw_pre", (300,)), ("dgate", (300,) if gate == "channel" else (45, 1)))}
        check_backward(t, h, before={k: v.clone() for k, v in first.items()}, accumulate=True, **first)


def test_rows_of_zeros_and_large_values():
    t = make(8, 256, "fp32")
    for k in ("x", "y"):
        t[k][2] = 0.0
        t[k][3] *= 1e15
        t[k][4] *= 1e-15
    h, _ = check_forward(t)
    got = check_backward(t, h)
    assert all(bool(torch.isfinite(v).all()) for v in got.values())


def test_a_row_of_nan_stays_alone():
    t = make(30, 512, "bf16")
    h, u = check_forward(t)
    t["y"][7] = float("nan")
    h2, u2 = dgr.block_norm(t["x"], t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9, w_pre=t["w_pre"], eps=1e-5)
    keep = torch.arange(30, device="cuda") != 7
    assert torch.equal(h2[keep], h[keep]) and torch.equal(u2[keep], u[keep])
    assert bool(torch.isnan(h2[7]).all()) and bool(torch.isnan(u2[7]).all())


def test_no_tokens():
    t = make(0, 64, "bf16")
    h, u = dgr.block_norm(t["x"], t["y"], w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    assert h.shape == u.shape == (0, 64)
    outs = {k: torch.full((64,), 3.0, device="cuda") for k in ("dw_post", "dgate", "dw_pre")}
    dgr.block_norm_backward(h, t["y"], t["dh"], t["du"], w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"],
                            accumulate=True, **outs)
    assert all(bool((v == 3.0).all()) for v in outs.values())
    dgr.block_norm_backward(h, t["y"], t["dh"], t["du"], w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"], **outs)
    assert all(bool((v == 0.0).all()) for v in outs.values())


def test_rows_past_2_to_the_31_elements():
    T, H, ld = 3, 96, (1 << 30) + 8
    t = make(T, H, "bf16")
    for k in ("x", "y", "dh", "du"):
        wide = torch.empty((T - 1) * ld + H, dtype=torch.bfloat16, device="cuda").as_strided((T, H), (ld, 1))
        wide.copy_(t[k])
        t[k] = wide
    h, _ = check_forward(t)
    check_backward(t, h)


def _call(t, alpha=0.9):
    h, u = dgr.block_norm(t["x"], t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=alpha, w_pre=t["w_pre"])
    g = dgr.block_norm_backward(h, t["y"], t["dh"], t["du"], w_post=t["w_post"], gate=t["gate"], res_scale=alpha,
                                w_pre=t["w_pre"])
    return torch.cat([h.float().reshape(-1), u.float().reshape(-1)] + [g[k].float().reshape(-1) for k in sorted(g)])


@pytest.mark.parametrize("T,H,dtype,gate", [(1500, 264, "bf16", "token"), (900, 2048, "bf16", "channel"),
                                            (700, 1000, "fp32", "channel")])
def test_no_schedule_changes_a_bit(T, H, dtype, gate):
    t = make(T, H, dtype, gate)
    base = bits(_call(t))
    for sch in SCHEDULES:
        with schedule(*sch):
            assert (bits(_call(t)) == base).all(), sch
    assert (assert_replays_identical(lambda: _call(t), n=6) == base).all()


def test_another_stream_and_a_captured_graph():
    t = make(400, 1024, "bf16")
    want = _call(t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        busy = busy @ busy * 1e-3
    ws = dgr.workspace(dgr.block_norm_workspace_bytes(400, 1024))
    torch.cuda.synchronize()
    h, u = dgr.block_norm(t["x"], t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9, w_pre=t["w_pre"], stream=side)
    g = dgr.block_norm_backward(h, t["y"], t["dh"], t["du"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9,
                                w_pre=t["w_pre"], ws=ws, stream=side)
    side.synchronize()
    got = torch.cat([h.float().reshape(-1), u.float().reshape(-1)] + [g[k].float().reshape(-1) for k in sorted(g)])
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgr.block_norm(t["x"], t["y"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9, w_pre=t["w_pre"], h=h, u=u)
        dgr.block_norm_backward(h, t["y"], t["dh"], t["du"], w_post=t["w_post"], gate=t["gate"], res_scale=0.9,
                                w_pre=t["w_pre"], ws=ws, **g)
    for v in (h, u, *g.values()):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = torch.cat([h.float().reshape(-1), u.float().reshape(-1)] + [g[k].float().reshape(-1) for k in sorted(g)])
    assert torch.equal(got, want)
