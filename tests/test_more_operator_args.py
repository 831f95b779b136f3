"""What the gated feed-forward, the norm and rotation of queries and keys and the token log probabilities
refuse, on the host and before any launch (these calls never reach a device)."""
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


def at(n, off):
    return ctypes.c_void_p((n << 32) + off)


def test_workspace_sizes(L):
    assert dgr.gated_ffn_workspace_bytes(1, 8, 8, 1) >= 256
    for bad in ((-1, 8, 8, 1), (1, 0, 8, 1), (1, 8, 0, 1), (1, 8, 8, 0), (1, 8, 8, 1025), (1 << 31, 8, 8, 1)):
        assert dgr.gated_ffn_workspace_bytes(*bad) == 0
    assert dgr.qk_norm_rope_workspace_bytes(100, 8, 2, 128) > 2 * 128 * 4
    for bad in ((-1, 8, 2, 128), (1, 0, 0, 128), (1, 8, 2, 514), (1, 1025, 1, 64), (1, -1, 2, 64)):
        assert dgr.qk_norm_rope_workspace_bytes(*bad) == 0
    assert dgr.token_logprobs_workspace_bytes(100) >= 256 and dgr.token_logprobs_workspace_bytes(-1) == 0


def test_gated_ffn(L):
    ok = dict(x=P(1), ldx=64, wg=P(2), wu=P(3), offs=P(4), E=2, T=10, H=64, F=32, act=0, h=P(5), ldh=32, g=P(6), ldg=32,
              u=P(7), ldu=32, ws=P(8), n=256, s=None)

    def call(**kw):
        return L.dgr_gated_ffn(*{**ok, **kw}.values())

    for kw in (dict(T=-1), dict(H=0), dict(F=0), dict(E=0), dict(act=2), dict(act=-1), dict(offs=None), dict(x=None), dict(wg=None),
               dict(wu=None), dict(h=None), dict(ws=None), dict(ldx=63), dict(ldh=31), dict(ldg=24), dict(ldu=24)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(T=(1 << 31) - 1), dict(E=1025), dict(H=(1 << 20) + 8, ldx=BIG), dict(F=(1 << 20) + 8),
               dict(H=1 << 20, ldx=BIG, F=1 << 19, ldh=BIG, ldg=BIG, ldu=BIG)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(H=60), dict(F=28), dict(ldx=68), dict(ldh=36), dict(x=at(1, 8)), dict(wg=at(2, 2)), dict(wu=at(3, 8)), dict(h=at(5, 8)),
               dict(g=at(6, 4)), dict(offs=at(4, 4)), dict(ws=at(8, 128))):
        assert call(**kw) == MISALIGNED, kw
    assert call(n=255) == TOO_SMALL
    for kw in (dict(h=P(1)), dict(h=P(2)), dict(g=P(3)), dict(u=P(4)), dict(g=P(5)), dict(u=at(5, 64)), dict(h=P(8)), dict(ws=P(1)), dict(ws=P(2))):
        assert call(**kw) == ALIAS, kw


def test_gated_ffn_backward(L):
    ok = dict(dh=P(1), lddh=32, g=P(2), ldg=32, u=P(3), ldu=32, wg=P(4), wu=P(5), offs=P(6), E=2, T=10, H=64, F=32, act=1, dg=P(7),
              lddg=32, du=P(8), lddu=32, dx=P(9), lddx=64, ws=P(10), n=512, s=None)

    def call(**kw):
        return L.dgr_gated_ffn_backward(*{**ok, **kw}.values())

    for kw in (dict(dh=None), dict(g=None), dict(u=None), dict(dg=None), dict(du=None), dict(wg=None), dict(wu=None), dict(ws=None),
               dict(lddh=31), dict(lddx=56), dict(lddg=24), dict(act=7), dict(offs=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(lddh=36), dict(dx=at(9, 8)), dict(dg=at(7, 8)), dict(wu=at(5, 8)), dict(u=at(3, 2))):
        assert call(**kw) == MISALIGNED, kw
    assert call(n=511) == TOO_SMALL
    for kw in (dict(dx=P(1)), dict(dx=P(7)), dict(dg=P(1)), dict(dg=P(3)), dict(du=P(2)), dict(dg=P(2), lddg=64), dict(dx=P(4)), dict(du=P(6)),
               dict(dg=P(8)), dict(ws=P(1)), dict(ws=P(5)), dict(dx=P(10))):
        assert call(**kw) == ALIAS, kw


QK = dict(q=P(1), qt=256, qh=64, nq=4, k=P(2), kt=128, kh=64, nk=2, dt=1, T=10, D=64, wq=P(3), wk=P(4), wdt=1, cos=P(5), sin=P(6), P_=100,
          R=32, inter=0, pos=P(7), eps=1e-6)


def test_qk_norm_rope(L):
    ok = dict(QK, qo=P(8), qot=256, qoh=64, ko=P(9), kot=128, koh=64, ws=P(10), n=256, s=None)

    def call(**kw):
        return L.dgr_qk_norm_rope(*{**ok, **kw}.values())

    for kw in (dict(dt=2), dict(wdt=3), dict(T=-1), dict(D=0), dict(D=63), dict(R=0), dict(R=31), dict(R=66), dict(P_=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(nq=-1), dict(nq=0, nk=0), dict(ws=None), dict(q=None), dict(ko=None), dict(cos=None), dict(pos=None),
               dict(qh=63), dict(qt=63), dict(qoh=60), dict(qt=128), dict(kot=64)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(T=(1 << 26) + 1), dict(D=514, qt=BIG, qh=514, kt=BIG, kh=514, qot=BIG, qoh=514, kot=BIG, koh=514), dict(nq=1025)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=at(1, 1)), dict(wq=at(3, 1)), dict(cos=at(5, 2)), dict(pos=at(7, 2)), dict(ws=at(10, 64)), dict(dt=0, ko=at(9, 2))):
        assert call(**kw) == MISALIGNED, kw
    assert call(n=255) == TOO_SMALL
    for kw in (dict(qo=P(2)), dict(ko=P(1)), dict(ko=P(8)), dict(qo=P(5)), dict(ko=P(4)), dict(qo=at(1, 128)), dict(qo=P(1), qot=320),
               dict(ws=P(1)), dict(ws=P(7)), dict(qo=P(10)), dict(q=P(1), qt=512, k=at(1, 256), kt=512, qo=P(1), qot=512, ko=at(1, 384), kot=512)):
        assert call(**kw) == ALIAS, kw


def test_qk_norm_rope_backward(L):
    ok = dict(dqo=P(11), dqot=256, dqoh=64, dko=P(12), dkot=128, dkoh=64, **QK, dq=P(13), dqt=256, dqh=64, dk=P(14), dkt=128, dkh=64,
              dwq=P(15), dwk=P(16), acc=0, ws=P(17), n=BIG, s=None)

    def call(**kw):
        return L.dgr_qk_norm_rope_backward(*{**ok, **kw}.values())

    for kw in (dict(dqo=None), dict(dk=None), dict(wq=None), dict(nk=0), dict(dqt=64), dict(ws=None)):
        assert call(**kw) == INVALID, kw
    assert call(n=256) == TOO_SMALL
    for kw in (dict(dwq=at(15, 2)), dict(dq=at(13, 1))):
        assert call(**kw) == MISALIGNED, kw
    for kw in (dict(dq=P(1)), dict(dq=P(12)), dict(dk=P(13)), dict(dwq=P(3)), dict(dwk=P(15)), dict(dwq=P(17)), dict(dq=P(11), dqt=512),
               dict(dwk=P(14)), dict(ws=P(11))):
        assert call(**kw) == ALIAS, kw


def test_token_logprobs(L):
    ok = dict(z=P(1), dt=1, T=10, V=100, ld=100, ids=P(2), tau=1.0, K=5, logp=P(3), H=P(4), lse=P(5), st=P(6), ti=P(7), tz=P(8), tp=P(9), ws=P(10),
              n=256, s=None)

    def call(**kw):
        return L.dgr_token_logprobs(*{**ok, **kw}.values())

    for kw in (dict(dt=2), dict(T=-1), dict(V=0), dict(ld=99), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")),
               dict(z=None), dict(ids=None), dict(K=-1), dict(K=0), dict(ti=None, tz=None, tp=None), dict(ws=None),
               dict(K=0, logp=None, H=None, lse=None, st=None, ti=None, tz=None, tp=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(K=129), dict(V=(1 << 20) + 1, ld=BIG), dict(T=(1 << 26) + 1), dict(tau=1e-7), dict(tau=1e7)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(z=at(1, 1)), dict(ids=at(2, 2)), dict(tp=at(9, 2)), dict(ws=at(10, 8))):
        assert call(**kw) == MISALIGNED, kw
    assert call(n=100) == TOO_SMALL
    for kw in (dict(logp=P(1)), dict(H=P(2)), dict(lse=P(3)), dict(tp=P(8)), dict(st=at(5, 4)), dict(ws=P(1)), dict(ti=P(10))):
        assert call(**kw) == ALIAS, kw


def test_token_logprobs_backward(L):
    ok = dict(z=P(1), dt=0, T=10, V=100, ld=104, ids=P(2), tau=1.0, st=P(3), H=P(4), dl=P(5), dH=P(6), dz=P(7), ldd=100, s=None)

    def call(**kw):
        return L.dgr_token_logprobs_backward(*{**ok, **kw}.values())

    for kw in (dict(st=None), dict(dz=None), dict(dl=None, dH=None), dict(ids=None), dict(H=None), dict(ldd=99), dict(tau=0.0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dz=at(7, 2)), dict(dl=at(5, 1))):
        assert call(**kw) == MISALIGNED, kw
    for kw in (dict(dz=P(1)), dict(dz=at(1, 16), ldd=104), dict(dz=P(3)), dict(dz=P(6))):
        assert call(**kw) == ALIAS, kw


def test_binding_checks_shapes_and_types():
    bf = torch.bfloat16
    x, w, h = torch.zeros(4, 8, dtype=bf), torch.zeros(2, 16, 8, dtype=bf), torch.zeros(4, 16, dtype=bf)
    offs = torch.zeros(3, dtype=torch.int64)
    for bad in (dict(act="tanh"), dict(offs=None), dict(offs=offs[:2]), dict(offs=offs.int()), dict(h=h.float()), dict(gate=h[:, :8])):
        with pytest.raises(ValueError):
            dgr.gated_ffn(x, w, w, **{**dict(offs=offs, h=h, ws=x), **bad})
    with pytest.raises(TypeError):
        dgr.gated_ffn(x, w.float(), w.float(), offs=offs)
    with pytest.raises(ValueError):
        dgr.gated_ffn(x, w, w[:1], offs=offs)
    with pytest.raises(ValueError):
        dgr.gated_ffn(x.t(), w, w, offs=offs)
    with pytest.raises(ValueError):
        dgr.gated_ffn_backward(h, h, h, w, w, offs=offs, dw_gate=torch.zeros(2, 16, 8))
    with pytest.raises(ValueError):  # sizes that the grouped weight gradient does not take
        dgr.gated_ffn_backward(h, h, h, w, w, offs=offs, x=x, dw_gate=torch.zeros(2, 16, 8))
    q, c, pos = torch.zeros(4, 2, 8), torch.zeros(5, 4), torch.zeros(4, dtype=torch.int32)
    for bad in (dict(q=q[0]), dict(q=None), dict(cos=c[0]), dict(sin=c[:, :2]), dict(positions=pos.long()), dict(positions=pos[:2]),
                dict(w_q=torch.ones(7)), dict(w_q=torch.ones(8), w_k=torch.ones(8, dtype=bf)), dict(q_out=q.to(bf)), dict(k=q.to(bf))):
        with pytest.raises(ValueError):
            dgr.qk_norm_rope(**{**dict(q=q, k=None, cos=c, sin=c, positions=pos, q_out=q, ws=q), **bad})
    with pytest.raises(ValueError):
        dgr.qk_norm_rope_backward(q, None, q, None, c, c, pos, w_q=torch.ones(8), accumulate=True)
    with pytest.raises(ValueError):
        dgr.qk_norm_rope_backward(q, q, q, None, c, c, pos)
    z, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    for bad in (dict(ids=ids.long()), dict(ids=ids[:3]), dict(logits=z.t()[:4]), dict(logits=z[0]), dict(top=-1), dict(logp=z), dict(stats=z[:, :2])):
        with pytest.raises(ValueError):
            dgr.token_logprobs(**{**dict(logits=z, ids=ids, ws=z), **bad})
    with pytest.raises(TypeError):
        dgr.token_logprobs(z.half(), ids, ws=z)
    with pytest.raises(ValueError):
        dgr.token_logprobs_backward(z, ids, z, dlogp=z[:, 0].clone())
