"""Gradients of the norm of heads close to zero, with nothing (eps = 0) or little beside their mean square."""
import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr
import more_operator_ref as ref
from test_gpu_qk_norm_rope import angles, make

pytestmark = pytest.mark.gpu

QUANTUM = 2.0 ** -149  # between subnormal numbers of binary32


def near(got, want, bound, what):
    err = (ref.d(got) - want).abs()
    assert got.isfinite().all() and (err <= bound).all(), (what, float((err / bound).max()))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,R", [(64, 64), (128, 64), (20, 8), (42, 20)])
@pytest.mark.parametrize("scale,eps", [(1.0, 0.0), (1e-12, 0.0), (4e-20, 0.0), (1e-20, 0.0), (1e-20, 1e-38)])
def test_heads_close_to_zero(scale, eps, D, R, dtype, inter):
    """r^2 leaves the range of binary32 from |v| of 5e-20 down, r and the gradient do not."""
    t, dy = make(9, 4, 2, D, R, dtype)
    for n in "qk":
        t[n] = (ref.d(t[n]) * scale).to(t[n].dtype).cuda()
    got = dgr.qk_norm_rope_backward(*dy, **t, eps=eps, interleaved=inter)
    c, s = angles(t)
    for n, g in zip("qk", dy):
        v = ref.d(t[n])
        args = ref.d(g), v, ref.d(t["w_" + n]), c, s, eps, inter
        (dv, dw), (bv, bw) = ref.qk_grads(*args), ref.qk_grad_bounds(*args, g.dtype)
        # squares, their mean and an eps that are subnormal lose half a quantum each: 3 halves of one of the mean (the D
        # squares' half quanta are divided by D), relative to it half as much of r and of dw, 3 / 2 of r^3
        mean = (v * v).mean(-1, keepdim=True) + eps
        lost = 1.5 * QUANTUM / mean
        r = 1 / torch.sqrt(mean)
        turned = ref.turn(ref.d(g).abs(), c.abs(), s.abs(), inter).abs() + ref.turn(ref.d(g).abs(), c.abs(), -s.abs(), inter).abs()
        w = ref.d(t["w_" + n]).abs()
        size = r * turned * w + v.abs() * r ** 3 / D * (turned * w * v.abs()).sum(-1, keepdim=True)
        near(got["d" + n], dv, bv + 1.5 * lost * size, "d" + n)
        near(got["dw_" + n], dw, bw + (0.5 * lost * turned * v.abs() * r).sum((0, 1)), "dw_" + n)
