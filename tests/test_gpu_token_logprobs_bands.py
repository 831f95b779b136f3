"""Lists of rows whose large logits lie side by side: a run of tokens that a mask leaves over, or that is above
the others, is in the shares of few threads, and of one CTA where a row has several."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import more_operator_ref as ref
from gpu_util import assert_replays_identical
from test_gpu_schedule import schedule
from test_gpu_token_logprobs import DT, INF, check_forward, make

pytestmark = pytest.mark.gpu

# rows, vocabulary, where the run starts: 8, 4 and 2 CTAs a row, and one
FORMS = [(1, 65536, 1000), (3, 131072, 70001), (5, 65600, 8191), (40, 20000, 2500), (20, 9001, 0), (160, 9001, 3000)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [513, 800, 1016])
@pytest.mark.parametrize("T,V,at", FORMS)
def test_band(T, V, at, n, dtype):
    for around in (-INF, 0.0):
        z, _ = make(T, V, dtype)
        band = z[:, at:at + n].clone()
        if around == -INF:
            z.fill_(-INF)
        z[:, at:at + n] = band + 20
        for K in (65, 100, 128):
            check_forward(z, None, top=K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [9000, 17000, 65600])
def test_ascending(V, dtype):
    """Every element larger than those before it, as far as the type holds that."""
    for T in (1, 7):
        z = torch.linspace(-8, 8, V).repeat(T, 1).to(DT[dtype]).cuda()
        for K in (1, 100, 128):
            check_forward(z, None, top=K)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_one_after_another(dtype):
    """Runs of every length in rows that the same CTAs take in turn: nothing of one row's is left for the next."""
    T, V = 24, 33000
    z, _ = make(T, V, dtype)
    g = torch.Generator().manual_seed(3)
    for t in range(T):
        n, at = 100 + 70 * t, int(torch.randint(0, V - 2000, (1,), generator=g))
        if t % 3 == 0:
            z[t, :at], z[t, at + n:] = -INF, -INF
        elif t % 3 == 1:
            z[t, at:at + n] += 20
    for K in (5, 128):
        want = check_forward(z, None, top=K)
        for cap in (8, 24):
            with schedule(0, 0, cap):
                got = dgr.token_logprobs(z, None, top=K)
            assert all(torch.equal(got[k], want[k]) for k in want)
    assert_replays_identical(lambda: torch.cat([v.reshape(-1).float() for v in dgr.token_logprobs(z, None, top=128).values()]), n=4)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_two_bands_in_two_ctas(dtype):
    """Each within a CTA's space, and more together than a row's."""
    z, _ = make(2, 65536, dtype)
    for first in (100, 8300, 16500, 33000):
        z[:, first:first + 500] += 20
    check_forward(z, None, top=128)
    z[0, 20:60] = 50.0  # ties at the list's top
    got = check_forward(z, None, top=128)
    assert got["top_ids"][0, :40].tolist() == list(range(20, 60)) and ref.d(got["top_logits"])[0, 0] == 50
