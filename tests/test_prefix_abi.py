"""Refusals of prefix_attn, on the host (no GPU)."""
import ctypes

import pytest

import speculative_decoding_verification_packed_gb300 as svp
from speculative_decoding_verification_packed_gb300 import build as svp_build
from test_cache_abi import BAD_CACHES, cache

OK, INV, UNS, WSP = svp.SVP_OK, svp.SVP_EINVAL, svp.SVP_EUNSUPPORTED, svp.SVP_EWORKSPACE
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def L():
    svp_build.build()
    return svp.lib()


def heads(*a):
    return ctypes.byref(svp.svp_heads(*a))


def call(L, q=16, stride=512, ca=None, ctx=16, cu=16, n=1, m=4, w=4, groups=16, length=16, ng=1, h=None, dtype=1, out=16,
         ws=1 << 20, wsb=BIG):
    c = cache() if ca is None else ca
    return L.svp_prefix_attn(q, stride, ctypes.byref(c), ctx, cu, n, m, w, groups, length, ng,
                             heads(4, 2, 128, 0.0) if h is None else h, dtype, out, None, ws, wsb, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches(L, bad, status):
    assert call(L, ca=cache(**bad)) == status
    assert call(L, ca=cache(**bad), ng=0) == status


def test_refusals(L):
    nb, small = ctypes.c_size_t(0), ctypes.c_size_t(0)
    size = lambda h, dtype=1, m=4: L.svp_prefix_attn_workspace_size(h, dtype, m, ctypes.byref(nb))
    assert size(None) == INV and size(heads(4, 3, 128, 0.0)) == INV and size(heads(4, 2, 128, 0.0), m=-1) == INV
    assert size(heads(4, 2, 96, 0.0)) == UNS and size(heads(129, 1, 128, 0.0)) == UNS and size(heads(4, 2, 128, 0.0), 2) == UNS
    sizes = []
    for m in (0, 1, 4, 1000):
        assert size(heads(4, 2, 128, 0.0), m=m) == OK
        sizes.append(nb.value)
    assert L.svp_chunk_attn_workspace_size(heads(4, 2, 128, 0.0), 1, ctypes.byref(small)) == OK
    assert sizes == sorted(sizes) and sizes[0] >= small.value
    need = sizes[2]
    assert call(L, n=-1) == INV and call(L, m=-1) == INV and call(L, w=0) == INV and call(L, ng=-1) == INV
    assert call(L, q=None) == INV and call(L, ctx=None) == INV and call(L, cu=None) == INV and call(L, out=None) == INV
    assert call(L, groups=None) == INV and call(L, length=None) == INV
    assert call(L, q=24) == INV and call(L, out=8) == INV and call(L, stride=511) == INV and call(L, stride=516) == INV
    assert call(L, ws=(1 << 20) + 8) == INV
    assert call(L, n=1025) == UNS and call(L, ng=1025) == UNS and call(L, dtype=svp.SVP_F32) == UNS
    assert call(L, dtype=svp.SVP_E4M3) == UNS and call(L, h=heads(4, 2, 96, 0.0)) == UNS
    assert call(L, ws=None) == WSP and call(L, wsb=need - 1) == WSP
    assert call(L, n=0) == OK and call(L, m=0) == OK and call(L, n=0, groups=None, length=None) == OK
    assert call(L, ca=cache(dtype=svp.SVP_F32)) == UNS                # bf16 queries over an fp32 cache
    for scale in (-0.5, float("nan"), float("inf"), -float("inf")):
        assert call(L, h=heads(4, 2, 128, scale)) == INV
