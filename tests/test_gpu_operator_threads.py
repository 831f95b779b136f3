"""Host threads that call one operator with different sizes (and so amounts of shared memory for one
kernel), each on a stream of its own: every call is taken and gives the results it gives alone."""
import sys
import threading

import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr

pytestmark = pytest.mark.gpu


def balance(G, E=512):
    g = torch.Generator(device="cuda").manual_seed(G)
    x = torch.randn(2048, E, generator=g, device="cuda")
    ids = torch.randint(0, E, (2048, 2), generator=g, device="cuda", dtype=torch.int32)
    offs = torch.arange(G + 1, device="cuda") * (2048 // G)
    ws = dgr.workspace(dgr.router_balance_workspace_bytes(2048, E, G))
    out = dict(loss=torch.empty(1, device="cuda"), counts=torch.empty(G, E, dtype=torch.int32, device="cuda"),
               tokens=torch.empty(G, dtype=torch.int32, device="cuda"), ws=ws)
    return lambda s: dgr.router_balance(x, ids, 0.1, offs=offs, stream=s, **out)


def norm(T, H=4096):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, y = torch.randn(T, H, generator=g, device="cuda"), torch.randn(T, H, generator=g, device="cuda")
    w, h, u = torch.ones(H, device="cuda"), torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    return lambda s: dgr.block_norm(x, y, w_post=w, w_pre=w, h=h, u=u, stream=s)


def norm_back(T, H=512):
    g = torch.Generator(device="cuda").manual_seed(T)
    h, y, dh, du = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(4))
    w, ws = torch.ones(H, device="cuda"), dgr.workspace(dgr.block_norm_workspace_bytes(T, H))
    out = dict(dx=torch.empty_like(h), dy=torch.empty_like(h), dw_post=torch.empty(H, device="cuda"),
               dw_pre=torch.empty(H, device="cuda"), ws=ws)
    return lambda s: list(dgr.block_norm_backward(h, y, dh, du, w_post=w, w_pre=w, stream=s, **out).values())


def distill(K, T=4, V=1 << 20):
    g = torch.Generator(device="cuda").manual_seed(K)
    z = torch.randn(T, V, generator=g, device="cuda")
    top = torch.randn(T, V, generator=g, device="cuda").topk(K, dim=1)
    ids, t, ws = top.indices.to(torch.int32), top.values.contiguous(), dgr.workspace(dgr.topk_distill_workspace_bytes(T))
    out = dict(loss=torch.empty(1, device="cuda"), row_loss=torch.empty(T, device="cuda"), ws=ws)
    return lambda s: dgr.topk_distill(z, ids, t, stream=s, **out)


@pytest.mark.parametrize("make,sizes", [(balance, (1, 1024)), (norm, (500, 2000)), (norm_back, (4000, 8000)), (distill, (1024, 512))],
                         ids=["balance", "norm", "norm backward", "distill"])
def test_threads(make, sizes):
    """Three threads a size, switched between as often as the interpreter can."""
    calls = [make(n) for n in sizes for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in calls]
    want = [[v.clone() for v in f(None)] for f in calls]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(calls))

    def work(i):
        start.wait()
        try:
            for _ in range(1500):
                got = calls[i](streams[i])
            streams[i].synchronize()
            wrong.extend(n for n, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    assert not wrong, wrong
