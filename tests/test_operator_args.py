"""What the router balance loss, the block norms and the distillation loss refuse, on the host and
before any launch (these calls never reach a device)."""
import ctypes

import pytest
import torch

import deterministic_gradient_reduction_gb300 as dgr

INVALID, UNSUPPORTED, TOO_SMALL, ALIAS, MISALIGNED = 1, 2, 3, 4, 5
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    dgr.build()
    return dgr.lib()


def P(n):
    return ctypes.c_void_p(n << 32)  # far apart; never read: every call fails its checks first


def test_workspace_sizes(L):
    assert dgr.router_balance_workspace_bytes(65536, 128) > 128 * 128 * 8
    assert dgr.router_balance_workspace_bytes(0, 1) >= 256
    for bad in ((-1, 8, 1), (8, 0, 1), (8, 1025, 1), (8, 8, 0), (8, 8, 1025), (1 << 31, 8, 1)):
        assert dgr.router_balance_workspace_bytes(*bad) == 0
    assert dgr.block_norm_workspace_bytes(16384, 4096) >= 256 + 152 * 2 * 4096 * 4
    for bad in ((-1, 8), (8, 0), (8, 16385), (1 << 31, 8)):
        assert dgr.block_norm_workspace_bytes(*bad) == 0
    assert dgr.topk_distill_workspace_bytes(100) >= 256 and dgr.topk_distill_workspace_bytes(-1) == 0


def test_router_balance(L):
    ok = dict(x=P(1), dt=0, N=100, E=16, ld=16, ids=P(2), K=2, ldi=2, mask=None, offs=None, G=1, score=0, coeff=1.0,
              counts=P(3), tokens=P(4), loss=P(5), ws=P(6), n=BIG, s=None)

    def call(**kw):
        return L.dgr_router_balance(*{**ok, **kw}.values())

    for kw in (dict(dt=2), dict(N=-1), dict(E=0), dict(K=0), dict(G=0), dict(ld=15), dict(ldi=1), dict(score=2),
               dict(score=-1), dict(G=2), dict(x=None), dict(ids=None), dict(counts=None), dict(tokens=None),
               dict(loss=None), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(N=1 << 31), dict(E=1025, ld=1025), dict(K=1025, ldi=1025), dict(G=1025, offs=P(7))):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=300) == TOO_SMALL
    for kw in (dict(x=ctypes.c_void_p(2)), dict(ids=ctypes.c_void_p(6)), dict(ws=ctypes.c_void_p(64)),
               dict(offs=ctypes.c_void_p(4)), dict(loss=ctypes.c_void_p(2))):
        assert call(**kw) == MISALIGNED, kw
    for kw in (dict(counts=P(1)), dict(tokens=P(2)), dict(loss=P(3)), dict(ws=P(1)), dict(loss=P(6))):
        assert call(**kw) == ALIAS, kw


def test_router_balance_backward(L):
    ok = dict(x=P(1), dt=1, N=100, E=16, ld=16, mask=None, offs=None, G=1, score=0, K=2, coeff=1.0, counts=P(3),
              tokens=P(4), dloss=None, dx=P(5), ldd=16, acc=0, s=None)

    def call(**kw):
        return L.dgr_router_balance_backward(*{**ok, **kw}.values())

    for kw in (dict(dt=9), dict(N=-1), dict(E=0), dict(K=0), dict(G=3), dict(ld=8), dict(ldd=8), dict(score=5),
               dict(x=None), dict(dx=None), dict(counts=None), dict(tokens=None)):
        assert call(**kw) == INVALID, kw
    assert call(E=1025, ld=1025, ldd=1025) == UNSUPPORTED
    assert call(x=ctypes.c_void_p(1)) == MISALIGNED and call(dx=ctypes.c_void_p(1)) == MISALIGNED
    for kw in (dict(dx=P(1)), dict(dx=P(3)), dict(dx=P(4)), dict(mask=P(5)), dict(dloss=P(5))):
        assert call(**kw) == ALIAS, kw


def test_block_norm(L):
    ok = dict(x=P(1), ldx=64, y=P(2), ldy=64, dt=1, T=10, H=64, w1=P(3), g=None, mode=0, w2=P(4), wdt=1, a=1.0, eps=1e-6,
              h=P(5), ldh=64, u=P(6), ldu=64, s=None)

    def call(**kw):
        return L.dgr_block_norm(*{**ok, **kw}.values())

    for kw in (dict(dt=2), dict(wdt=2), dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=float("nan")), dict(mode=3),
               dict(mode=1), dict(g=P(7)), dict(w2=None), dict(u=None), dict(h=None), dict(x=None), dict(ldx=63),
               dict(ldy=63), dict(ldh=63), dict(ldu=63), dict(y=None), dict(y=None, w1=None),
               dict(y=None, w1=None, h=None, a=0.5)):
        assert call(**kw) == INVALID, kw
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(H=16385, ldx=16385, ldy=16385, ldh=16385, ldu=16385) == UNSUPPORTED
    for kw in (dict(x=ctypes.c_void_p(3)), dict(w1=ctypes.c_void_p(1)), dict(u=ctypes.c_void_p(9))):
        assert call(**kw) == MISALIGNED, kw
    for kw in (dict(h=P(2)), dict(u=P(1)), dict(u=P(2)), dict(u=P(5)), dict(h=P(3)), dict(u=P(4)), dict(h=P(1), ldh=128),
               dict(h=ctypes.c_void_p((1 << 32) + 128))):
        assert call(**kw) == ALIAS, kw


def test_block_norm_backward(L):
    ok = dict(h=P(1), ldh=64, y=P(2), ldy=64, dh=P(3), lddh=64, du=P(4), lddu=64, dt=1, T=10, H=64, w1=P(5), g=P(6),
              mode=1, w2=P(7), wdt=0, a=1.0, eps=1e-6, dx=P(8), lddx=64, dy=P(9), lddy=64, dw1=P(10), dg=P(11),
              dw2=P(12), acc=0, ws=P(13), n=BIG, s=None)

    def call(**kw):
        return L.dgr_block_norm_backward(*{**ok, **kw}.values())

    for kw in (dict(dt=2), dict(T=-1), dict(H=0), dict(mode=0), dict(g=None), dict(du=None), dict(w2=None), dict(h=None),
               dict(dh=None, du=None, w2=None, dw2=None), dict(y=None), dict(dy=None), dict(dx=None),
               dict(w1=None), dict(g=None, mode=0), dict(ldh=1), dict(ldy=1), dict(lddh=1), dict(lddu=1), dict(lddx=1),
               dict(lddy=1), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    assert call(n=300) == TOO_SMALL
    for kw in (dict(dx=ctypes.c_void_p(1)), dict(dw1=ctypes.c_void_p(2)), dict(ws=ctypes.c_void_p(128)),
               dict(w2=ctypes.c_void_p(2))):
        assert call(**kw) == MISALIGNED, kw
    for kw in (dict(dx=P(1)), dict(dx=P(2)), dict(dx=P(4)), dict(dy=P(2)), dict(dy=P(8)), dict(dy=P(3)), dict(dw1=P(10), dw2=P(10)),
               dict(dg=P(6)), dict(ws=P(1)), dict(dx=P(3), lddx=128)):
        assert call(**kw) == ALIAS, kw


def test_topk_distill(L):
    ok = dict(z=P(1), dt=1, T=10, V=100, ld=100, ids=P(2), ldi=8, t=P(3), ldt=8, K=8, tau=1.0, lse=None, w=None, scale=1.0,
              dloss=None, rows=P(4), loss=P(5), dz=P(6), ldd=100, ws=P(7), n=256, s=None)

    def call(**kw):
        return L.dgr_topk_distill(*{**ok, **kw}.values())

    for kw in (dict(dt=2), dict(T=-1), dict(V=0), dict(K=0), dict(ld=99), dict(ldd=99), dict(ldi=7), dict(ldt=7),
               dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(z=None), dict(ids=None),
               dict(t=None), dict(rows=None), dict(rows=None, loss=None, dz=None), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    assert call(V=(1 << 20) + 1, ld=BIG, ldd=BIG) == UNSUPPORTED and call(K=1025, ldi=1025, ldt=1025) == UNSUPPORTED
    assert call(n=255) == TOO_SMALL
    for kw in (dict(z=ctypes.c_void_p(1)), dict(dz=ctypes.c_void_p(1)), dict(t=ctypes.c_void_p(2)), dict(ws=ctypes.c_void_p(8))):
        assert call(**kw) == MISALIGNED, kw
    for kw in (dict(dz=P(1), ldd=101), dict(dz=P(2)), dict(rows=P(3)), dict(loss=P(4)), dict(rows=P(6)), dict(ws=P(1)),
               dict(dz=ctypes.c_void_p((1 << 32) + 16))):
        assert call(**kw) == ALIAS, kw


def test_binding_checks_shapes_and_types():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dgr.router_balance(x, ids, 1.0, score="tanh")
    with pytest.raises(ValueError):
        dgr.router_balance(x, ids.long(), 1.0, loss=x[0, :1], counts=ids, tokens=ids, ws=x)
    with pytest.raises(ValueError):
        dgr.router_balance(x.t(), ids, 1.0)
    with pytest.raises(ValueError):
        dgr.router_balance(x, ids, 1.0, mask=torch.ones(3, dtype=torch.bool))
    with pytest.raises(ValueError):
        dgr.router_balance_backward(x, ids, ids, 2, 1.0, accumulate=True)
    with pytest.raises(ValueError):
        dgr.block_norm(x, x, w_post=torch.ones(7), h=x, u=x)
    with pytest.raises(ValueError):
        dgr.block_norm(x, x, gate=torch.ones(4, 2), h=x)
    with pytest.raises(ValueError):
        dgr.block_norm(x, x, w_post=torch.ones(8), w_pre=torch.ones(8).bfloat16(), h=x, u=x)
    with pytest.raises(ValueError):
        dgr.block_norm_backward(x, x, x, x, w_post=torch.ones(8), w_pre=torch.ones(8), accumulate=True)
    with pytest.raises(ValueError):
        dgr.topk_distill(x, ids.long(), x[:, :2], loss=x[0, :1], row_loss=x[:, 0].clone(), ws=x)
    with pytest.raises(ValueError):
        dgr.topk_distill(x, ids, torch.zeros(4, 3), loss=x[0, :1], row_loss=torch.zeros(4), ws=x)
    with pytest.raises(TypeError):
        dgr.topk_distill(x.half(), ids, torch.zeros(4, 2), loss=x[0, :1], row_loss=torch.zeros(4), ws=x)
