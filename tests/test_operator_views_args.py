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
