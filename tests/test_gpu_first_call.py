"""The products with tensor maps called from a host thread that has made no CUDA call before."""
import threading

import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import dgr_inputs as gi
from test_gpu_gated_ffn import make

pytestmark = pytest.mark.gpu


def _ffn():
    t = make([300, 1, 0, 200], 264, 520)
    ws, h = dgr.workspace(dgr.gated_ffn_workspace_bytes(501, 264, 520, 4)), torch.empty(501, 520, dtype=torch.bfloat16, device="cuda")
    return lambda s: [dgr.gated_ffn(t["x"], t["w_gate"], t["w_up"], offs=t["offs"], h=h, ws=ws, stream=s)]


def _dsrelu():
    d = gi.dsrelu_input(2, 256, 64, 256, seed=94, counts=[128, 128])
    a = [t.cuda() for t in (d.A, d.B, d.offs, d.dY)]
    ws, out = dgr.workspace(dgr.dsrelu_dprob_workspace_bytes(256, 256)), torch.empty(256, device="cuda")
    return lambda s: [dgr.dsrelu_dprob(*a, out, ws=ws, stream=s)]


@pytest.mark.parametrize("calls", [_ffn, _dsrelu], ids=["ffn", "dsrelu"])
def test_a_host_threads_first_call(calls):
    """A thread that has made no CUDA call before: the tensor maps need the device's context there too."""
    call, stream = calls(), torch.cuda.Stream()
    want = [v.clone() for v in call(None)]
    torch.cuda.synchronize()
    got = []

    def work():
        try:
            got.extend(call(stream))
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want)), got
