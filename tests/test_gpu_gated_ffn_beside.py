"""The gated feed-forward's backward of many rows beside a kernel of another stream that keeps part of the SMs: CTAs
that have no SM yet begin no tiles, and the elements of the others do not wait for that."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from test_gpu_gated_ffn import BF
from test_gpu_schedule import schedule

pytestmark = pytest.mark.gpu


def test_a_large_call_beside_another_streams_kernel():
    T, H, F, E, long = 32768, 2048, 4096, 8, 65536
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    w_gate, w_up = r(E, F, H) * H ** -0.5, r(E, F, H) * H ** -0.5
    dh, gate, up = r(T, F), r(T, F), r(T, F)
    offs = torch.arange(E + 1, device="cuda") * (T // E)
    ws, ws2 = (dgr.workspace(dgr.gated_ffn_workspace_bytes(long, H, F, E)) for _ in range(2))
    out = {k: torch.empty(T, n, dtype=BF, device="cuda") for k, n in (("dx", H), ("dgate", F), ("dup", F))}
    x, h = r(long, H), torch.empty(long, F, dtype=BF, device="cuda")
    here, other = torch.cuda.Stream(), torch.cuda.Stream()

    def timed():
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record(here)
        dgr.gated_ffn_backward(dh, gate, up, w_gate, w_up, offs=offs, ws=ws, stream=here, **out)
        b.record(here)
        return a, b

    def beside():
        with schedule(0, 0, 32):  # on 32 SMs, for some 7 ms
            dgr.gated_ffn(x, w_gate[0], w_up[0], h=h, ws=ws2, stream=other)
        pair = timed()
        end = torch.cuda.Event(enable_timing=True)
        end.record(other)
        torch.cuda.synchronize()
        return pair[0].elapsed_time(pair[1]), pair[0].elapsed_time(end)

    timed()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in out.items()}
    alone = []
    for _ in range(3):
        a, b = timed()
        torch.cuda.synchronize()
        alone.append(a.elapsed_time(b))
    took = [beside() for _ in range(3)]
    assert all(torch.equal(out[k], want[k]) for k in want) and dgr.read_device_status(ws) == 0
    # the CTAs that find no SM at first have their tiles when the others are done: twice the time, and
    # what the other kernel takes of memory and power
    ms, rest = min(took)
    assert rest > 3 * min(alone), "the other kernel did not last"
    assert ms < 3 * min(alone), (alone, took)
