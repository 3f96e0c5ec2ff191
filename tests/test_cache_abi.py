"""Refusals of the paged cache's calls, on the host (no GPU): every bad argument is answered
with a status before any CUDA call."""
import ctypes

import pytest

import speculative_decoding_verification_packed_gb300 as svp
from speculative_decoding_verification_packed_gb300 import build as svp_build

OK, INV, UNS, WSP = svp.SVP_OK, svp.SVP_EINVAL, svp.SVP_EUNSUPPORTED, svp.SVP_EWORKSPACE
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    svp_build.build()
    return svp.lib()


def cache(**kw):
    c = svp.svp_cache()
    c.k = c.v = 1 << 20
    c.k_exp = c.v_exp = 1 << 20
    c.block_table = 1 << 20
    c.max_pages, c.page_size, c.num_pages = 8, 16, 100
    c.stride_page, c.stride_head, c.stride_tok = 2 * 16 * 128, 16 * 128, 128
    c.dtype = svp.SVP_BF16
    for name, x in kw.items():
        setattr(c, name, x)
    return c


BAD_CACHES = [
    (dict(dtype=3), UNS), (dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=256), UNS),
    (dict(k=None), INV), (dict(v=None), INV), (dict(block_table=None), INV), (dict(max_pages=-1), INV),
    (dict(num_pages=-1), INV), (dict(num_pages=1 << 31), INV), (dict(max_pages=1 << 27), UNS),
    (dict(dtype=svp.SVP_E4M3, k_exp=None), INV), (dict(dtype=svp.SVP_E4M3, v_exp=(1 << 20) + 8), INV),
    (dict(k=(1 << 20) + 8), INV), (dict(stride_tok=64), INV), (dict(stride_head=0), INV),
    (dict(stride_page=-4096), INV), (dict(stride_tok=132), INV)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches(L, bad, status):
    c = cache(**bad)
    h = svp.svp_heads(4, 2, 128, 0.0)
    assert L.svp_cache_write(16, 16, 256, 1, ctypes.byref(c), 16, 16, None, 1, 4, 2, 128, 16, BIG, None) == status
    assert L.svp_cache_read(ctypes.byref(c), None, 16, 1, 4, 2, 128, 1, 16, 16, 16, BIG, None) == status
    assert L.svp_chunk_attn(16, 512, ctypes.byref(c), 16, 16, 1, 4, 4, ctypes.byref(h), 1, 16, None, 16, BIG,
                            None) == status


def test_write_refusals(L):
    c = cache()
    f = lambda k=16, v=16, stride=256, dtype=1, ca=ctypes.byref(c), ctx=16, cu=16, n=1, m=4, hkv=2, d=128, ws=16, \
        wsb=BIG: L.svp_cache_write(k, v, stride, dtype, ca, ctx, cu, None, n, m, hkv, d, ws, wsb, None)
    assert f(ca=None) == INV and f(n=-1) == INV and f(m=-1) == INV and f(hkv=0) == INV
    assert f(k=None) == INV and f(v=None) == INV and f(ctx=None) == INV and f(cu=None) == INV
    assert f(k=8) == INV and f(stride=255) == INV and f(stride=260) == INV
    assert f(d=96) == UNS and f(dtype=svp.SVP_E4M3) == UNS and f(dtype=9) == UNS
    assert f(ws=None) == WSP and f(wsb=64) == WSP
    assert f(n=0) == OK and f(m=0) == OK


def test_read_refusals(L):
    c = cache()
    f = lambda ca=ctypes.byref(c), cu=16, n=1, rows=4, hkv=2, d=128, dtype=1, k=16, v=16, ws=16, wsb=BIG: \
        L.svp_cache_read(ca, None, cu, n, rows, hkv, d, dtype, k, v, ws, wsb, None)
    assert f(ca=None) == INV and f(n=-1) == INV and f(rows=-1) == INV and f(hkv=-2) == INV
    assert f(cu=None) == INV and f(k=None) == INV and f(v=8) == INV
    assert f(d=32) == UNS and f(dtype=svp.SVP_E4M3) == UNS
    assert f(ws=None) == WSP and f(wsb=255) == WSP
    assert f(n=0) == OK and f(rows=0) == OK


def test_attention_refusals(L):
    c = cache()
    nb = ctypes.c_size_t(0)
    heads = lambda *a: ctypes.byref(svp.svp_heads(*a))
    assert L.svp_chunk_attn_workspace_size(heads(4, 3, 128, 0.0), 1, ctypes.byref(nb)) == INV
    assert L.svp_chunk_attn_workspace_size(heads(4, 2, 96, 0.0), 1, ctypes.byref(nb)) == UNS
    assert L.svp_chunk_attn_workspace_size(heads(129, 1, 128, 0.0), 1, ctypes.byref(nb)) == UNS
    assert L.svp_chunk_attn_workspace_size(heads(4, 2, 128, 0.0), svp.SVP_E4M3, ctypes.byref(nb)) == UNS
    assert L.svp_chunk_attn_workspace_size(None, 1, ctypes.byref(nb)) == INV
    assert L.svp_chunk_attn_workspace_size(heads(4, 2, 128, 0.0), 1, ctypes.byref(nb)) == OK
    need = nb.value
    assert need >= 256
    f = lambda q=16, stride=512, ca=ctypes.byref(c), ctx=16, cu=16, n=1, m=4, w=4, h=heads(4, 2, 128, 0.0), dtype=1, \
        out=16, ws=16, wsb=BIG: L.svp_chunk_attn(q, stride, ca, ctx, cu, n, m, w, h, dtype, out, None, ws, wsb, None)
    assert f(ca=None) == INV and f(h=None) == INV and f(n=-1) == INV and f(m=-1) == INV and f(w=0) == INV
    assert f(q=None) == INV and f(ctx=None) == INV and f(cu=None) == INV and f(out=None) == INV
    assert f(q=24) == INV and f(out=8) == INV and f(stride=511) == INV and f(stride=516) == INV
    assert f(n=1025) == UNS and f(dtype=svp.SVP_F32) == UNS and f(dtype=svp.SVP_E4M3) == UNS
    assert f(ws=None) == WSP and f(wsb=need - 1) == WSP
    assert f(n=0) == OK and f(m=0) == OK
    f32 = cache(dtype=svp.SVP_F32, stride_page=2 * 16 * 128, stride_head=16 * 128)
    assert f(ca=ctypes.byref(f32)) == UNS                       # bf16 queries over an fp32 cache
    for scale in (-0.5, float("nan"), float("inf"), -float("inf")):
        assert f(h=heads(4, 2, 128, scale)) == INV


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        svp.make_cache(x, x, torch.zeros(1, 2, dtype=torch.int32))
