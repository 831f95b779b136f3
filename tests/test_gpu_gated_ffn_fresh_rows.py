"""The gated feed-forward's backward of many rows multiplies rows of dgate and dup that other CTAs of the same launch
write. Called again and again with new gradients and the same buffers, dx comes of this call's rows, never of those
that the call before left there."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
from gpu_util import side_stream_contention
from test_gpu_gated_ffn import BF, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,H,F", [([5500, 4500], 1544, 72), ([4000, 1, 0, 6050], 1600, 264), ([10001], 1536, 1032)])
def test_rows_of_this_call(counts, H, F):
    t, T, E = make(counts, H, F), sum(counts), len(counts)
    ws = dgr.workspace(dgr.gated_ffn_workspace_bytes(T, H, F, E))
    out = {k: torch.empty(T, n, dtype=BF, device="cuda") for k, n in (("dx", H), ("dgate", F), ("dup", F))}
    side = torch.cuda.Stream()
    for i in range(24):
        t["dh"].copy_(torch.randn_like(t["dh"]))
        # pieces of few rows, where the elements come first in a launch of their own: a row's bits do not depend on its company
        want = []
        for e in range(E):
            for a in range(t["cuts"][e], t["cuts"][e + 1], 1000):
                part = [t[k][a:min(a + 1000, t["cuts"][e + 1])] for k in ("dh", "gate", "up")]
                want.append(dgr.gated_ffn_backward(*part, t["w_gate"][e], t["w_up"][e])["dx"])
        torch.cuda.synchronize()

        def call(stream):
            dgr.gated_ffn_backward(t["dh"], t["gate"], t["up"], t["w_gate"], t["w_up"], offs=t["offs"], ws=ws, stream=stream, **out)

        if i % 3 == 2:
            with side_stream_contention(2):
                call(side)
        else:
            call(side)
        torch.cuda.synchronize()
        assert torch.equal(out["dx"], torch.cat(want)), i
    assert dgr.read_device_status(ws) == 0
