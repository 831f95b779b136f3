"""The gated feed-forward, the norm and rotation and the token log probabilities called from several host threads
with different sizes, each on a stream of its own, and two calls at once on streams of different priorities: every
call gives the results it gives alone."""
import sys
import threading

import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from test_gpu_gated_ffn import make as make_ffn
from test_gpu_qk_norm_rope import make as make_qk
from test_gpu_token_logprobs import make as make_logits

pytestmark = pytest.mark.gpu


def ffn(counts, H, F):
    t, T, E = make_ffn(counts, H, F), sum(counts), len(counts)
    ws = dgr.workspace(dgr.gated_ffn_workspace_bytes(T, H, F, E))
    h = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    out = dict(dx=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), dgate=torch.empty_like(h), dup=torch.empty_like(h))
    w = dict(offs=t["offs"], ws=ws)

    def call(s):
        dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], h=h, stream=s, **w)
        dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], stream=s, **w, **out)
        return [h, *out.values()]

    return call


def qk(T, A, B, D, R, dtype):
    a, (dq, dk) = make_qk(T, A, B, D, R, dtype)
    ws = dgr.workspace(dgr.qk_norm_rope_workspace_bytes(T, A, B, D))
    f = [torch.empty_like(a["q"]), torch.empty_like(a["k"])]
    out = dict(dq=torch.empty_like(a["q"]), dk=torch.empty_like(a["k"]), dw_q=torch.empty(D, device="cuda"), dw_k=torch.empty(D, device="cuda"))

    def call(s):
        dgr.qk_norm_rope(**a, q_out=f[0], k_out=f[1], ws=ws, stream=s)
        dgr.qk_norm_rope_backward(dq, dk, **a, ws=ws, stream=s, **out)
        return f + list(out.values())

    return call


def logp(T, V, K, dtype):
    z, ids = make_logits(T, V, dtype)
    out = dict(dgr.token_logprobs(z, ids, top=K))
    ws, one, dz = dgr.workspace(256), torch.ones(T, device="cuda"), torch.empty(T, V, dtype=z.dtype, device="cuda")

    def call(s):
        dgr.token_logprobs(z, ids, top=K, ws=ws, stream=s, **out)
        dgr.token_logprobs_backward(z, ids, out["stats"], out["entropy"], dlogp=one, dentropy=one, dlogits=dz, stream=s)
        return [*out.values(), dz]

    return call


CALLS = {
    "ffn": (ffn, [([5500, 4500], 1544, 264), ([5000, 5200], 1544, 520), ([300, 1, 0, 200], 264, 520), ([3], 512, 1024)]),
    "qk": (qk, [(3000, 8, 2, 128, 128, "bf16"), (500, 4, 4, 256, 128, "fp32"), (70, 3, 1, 80, 80, "bf16"), (2000, 2, 2, 6, 6, "fp32")]),
    "logp": (logp, [(3, 70000, 128, "bf16"), (1300, 2000, 5, "bf16"), (300, 9001, 64, "fp32"), (40, 5000, 0, "fp32")]),
}


@pytest.mark.parametrize("name", CALLS)
def test_threads(name):
    make, sizes = CALLS[name]
    calls = [make(*n) for n in sizes for _ in range(2)]
    streams = [torch.cuda.Stream(priority=-(i % 2)) for i in range(len(calls))]
    want = [[v.clone() for v in f(None)] for f in calls]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(calls))

    def work(i):
        start.wait()
        try:
            for _ in range(200):
                got = calls[i](streams[i])
            streams[i].synchronize()
            wrong.extend((i, n) for n, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not wrong, wrong


def test_two_large_backward_calls_share_the_gpu():
    """Rows that one CTA multiplies are made by any other: neither call may wait for CTAs that have no SM yet."""
    calls = [ffn([5500, 4500], 1544, 264), ffn([9000, 1200], 1544, 264)]
    want = [[v.clone() for v in f(None)] for f in calls]
    low, high, other = torch.cuda.Stream(), torch.cuda.Stream(priority=-1), torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(other):
            y = x @ x  # has the SMs when the two arrive
        got = [calls[0](low), calls[1](high)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert y.isfinite().all()
