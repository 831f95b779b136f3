"""Tensors of one call that have elements in common, between one another's rows or heads, are refused on the host
before any launch (these calls never reach a device)."""
import pytest

import deterministic_gradient_reduction_gb300 as dgr
from test_more_operator_args import QK, P, at

ALIAS = 4


@pytest.fixture(scope="module")
def L():
    dgr.build()
    return dgr.lib()


def test_heads(L):
    """Heads of 64 bf16 (128 bytes) every 384 bytes, tokens every 1536; queries at 0, keys elsewhere in the row."""
    ok = dict(QK, qt=768, qh=192, k=at(1, 128), kt=768, kh=192, nk=4, qo=P(8), qot=256, qoh=64, ko=P(9), kot=256, koh=64, ws=P(10), n=256, s=None)

    def call(**kw):
        return L.dgr_qk_norm_rope(*{**ok, **kw}.values())

    for kw in (
            dict(qo=at(1, 2), qot=768, qoh=192),                # all but one element of its own input
            dict(qo=at(1, 126), qot=768, qoh=192),              # its last element
            dict(qo=at(1, 130), qot=768, qoh=192),              # the keys
            dict(qo=at(1, 256 + 1536 * 3 + 130), qot=768, qoh=192),  # the next head's query, three tokens on
            dict(qo=at(1, 256), qot=768, qoh=64),               # the row's gaps, at another distance
            dict(qo=at(1, 256), qot=960, qoh=192),
            dict(ko=at(8, 64)),                                 # the other output
            dict(T=1, qo=at(1, 64), qot=768, qoh=192), dict(T=1, qo=at(1, 256), qot=768, qoh=64),
            dict(nq=1, qh=7, qo=at(1, 64), qoh=9, qot=768),     # one head: its distance says nothing
            # [heads, 2, tokens, 64] with the tokens' runs of 1280 bytes shifted into one another
            dict(qt=64, qh=1280, k=P(2), kt=64, kh=64 * 10, qo=at(1, 1152), qot=64, qoh=1280)):
        assert call(**kw) == ALIAS, kw


def test_rows(L):
    """Rows of 40 bf16 (80 bytes) side by side in rows of 160: what reaches into its neighbour's."""
    ok = dict(x=P(1), ldx=64, wg=P(2), wu=P(3), offs=P(4), E=2, T=10, H=64, F=40, act=0, h=P(5), ldh=80, g=P(6), ldg=80,
              u=at(6, 80), ldu=80, ws=P(8), n=256, s=None)

    def forward(**kw):
        return L.dgr_gated_ffn(*{**ok, **kw}.values())

    for kw in (dict(u=at(6, 64)), dict(u=at(6, 96)), dict(u=at(6, 160 * 5 + 64)), dict(u=P(6)), dict(u=at(6, 80), ldu=88), dict(h=at(6, 160)),
               dict(h=at(6, 32)), dict(h=at(1, 80), ldh=64), dict(T=1, u=at(6, 64)), dict(h=at(6, 160 * 9 + 64), ldh=400)):
        assert forward(**kw) == ALIAS, kw
    ok_back = dict(dh=P(1), lddh=40, g=P(2), ldg=80, u=at(2, 80), ldu=80, wg=P(4), wu=P(5), offs=P(6), E=2, T=10, H=64, F=40, act=1, dg=P(7),
                   lddg=80, du=at(7, 80), lddu=80, dx=P(9), lddx=64, ws=P(10), n=512, s=None)

    def backward(**kw):
        return L.dgr_gated_ffn_backward(*{**ok_back, **kw}.values())

    for kw in (dict(du=at(7, 64)), dict(du=at(7, 96)), dict(dg=at(2, 80)), dict(dg=at(2, 16)), dict(dx=at(7, 160), lddx=80), dict(dx=at(2, 80), lddx=80),
               dict(dg=P(2), lddg=88)):
        assert backward(**kw) == ALIAS, kw
    back = dict(z=P(1), dt=0, T=10, V=100, ld=208, ids=P(2), tau=1.0, st=P(3), H=P(4), dl=P(5), dH=P(6), dz=at(1, 400), ldd=208, s=None)
    for kw in (dict(dz=at(1, 396)), dict(dz=at(1, 436)), dict(dz=at(1, 400 + 3 * 832 + 36)), dict(ldd=209)):
        assert L.dgr_token_logprobs_backward(*{**back, **kw}.values()) == ALIAS, kw
