"""The 64-bit forms' gradients against finite differences."""
import pytest
import torch

import more_operator_ref as ref


def difference(f, v, direction, h=1e-6):
    return float((f(v + h * direction) - f(v - h * direction)) / (2 * h))


def close(a, b):
    assert abs(a - b) <= 1e-7 * (1 + abs(b)), (a, b)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn(act):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w1, w2, dh, offs = r(7, 5), r(3, 4, 5), r(3, 4, 5), r(7, 4), [0, 2, 2, 7]
    _, a, b = ref.ffn(x, w1, w2, offs, act)
    da, db = ref.pre_grads(dh, a, b, act)
    got = ref.dx(da, db, w1, w2, offs)
    v = r(7, 5)
    close(difference(lambda t: (ref.ffn(t, w1, w2, offs, act)[0] * dh).sum(), x, v), float((got * v).sum()))
    if act == "gelu":
        assert torch.allclose(ref.activation(a, act), torch.nn.functional.gelu(a, approximate="tanh"), atol=1e-12)
    else:
        assert torch.allclose(ref.activation(a, act), torch.nn.functional.silu(a), atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qk(interleaved):
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    v, w, dy, ang = r(3, 2, 10), r(10), r(3, 2, 10), r(3, 3)
    c, s = torch.cos(ang), torch.sin(ang)
    dv, dw = ref.qk_grads(dy, v, w, c, s, 1e-3, interleaved)
    e, f = r(3, 2, 10), r(10)
    close(difference(lambda t: (ref.qk(t, w, c, s, 1e-3, interleaved) * dy).sum(), v, e), float((dv * e).sum()))
    close(difference(lambda t: (ref.qk(v, t, c, s, 1e-3, interleaved) * dy).sum(), w, f), float((dw * f).sum()))
    # a rotation keeps the length of every pair
    assert torch.allclose(ref.turn(v, c, s, interleaved).norm(dim=-1), v.norm(dim=-1))


def test_logp():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    z, ids, a, b, tau = 2 * r(4, 9), torch.tensor([3, -1, 0, 8]), r(4), r(4), 1.7
    z[2, 5] = -float("inf")

    def total(t):
        lp, H, _ = ref.logp_rows(t, tau)
        on = ids >= 0
        return (a[on] * lp[on, ids[on]]).sum() + (b[on] * H[on]).sum()

    got = ref.logp_grad(z, ids, a, b, tau)
    v = r(4, 9)
    v[2, 5] = 0
    close(difference(total, z, v), float((got * v).sum()))
    assert not got[1].any() and float(got[2, 5]) == 0
    lp, H, lse = ref.logp_rows(torch.full((1, 4), -float("inf"), dtype=torch.float64), 1.0)
    assert float(H) == 0 and float(lse) == -float("inf")
