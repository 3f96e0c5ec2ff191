"""Refusals of the pages' calls, on the host (no GPU)."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from speculative_decoding_verification_packed_gb300 import build as svp_build

OK, INV, UNS, WSP = svp.SVP_OK, svp.SVP_EINVAL, svp.SVP_EUNSUPPORTED, svp.SVP_EWORKSPACE
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def L():
    svp_build.build()
    return svp.lib()


def pages(**kw):
    p = svp.svp_pages()
    p.block_table = p.used = p.refs = 1 << 20
    p.n, p.max_pages, p.page_size, p.num_pages = 4, 8, 16, 100
    for name, x in kw.items():
        setattr(p, name, x)
    return ctypes.byref(p)


def caches(count=1, **kw):
    arr = (svp.svp_cache * max(count, 1))()
    for c in arr:
        c.k = c.v = c.block_table = 1 << 20
        c.max_pages, c.page_size, c.num_pages = 8, 16, 100
        c.stride_page, c.stride_head, c.stride_tok, c.dtype = 2 * 16 * 128, 16 * 128, 128, svp.SVP_BF16
    for name, x in kw.items():
        setattr(arr[count - 1], name, x)
    return arr


BAD = [(dict(n=-1), INV), (dict(max_pages=-1), INV), (dict(num_pages=-1), INV), (dict(num_pages=1 << 31), INV),
       (dict(page_size=8), UNS), (dict(page_size=256), UNS), (dict(n=1025), UNS), (dict(max_pages=1 << 27), UNS),
       (dict(n=1024, max_pages=1 << 22), UNS)]


def test_bad_pages(L):
    nb = ctypes.c_size_t(0)
    assert L.svp_pages_workspace_size(None, ctypes.byref(nb)) == INV
    assert L.svp_pages_workspace_size(pages(), None) == INV
    for bad, status in BAD:
        assert L.svp_pages_workspace_size(pages(**bad), ctypes.byref(nb)) == status
        assert L.svp_pages_resize(pages(**bad), 16, 1 << 20, BIG, None) == status
        assert L.svp_pages_fork(pages(**bad), caches(), 1, 2, 128, 16, 16, 16, 1, 1 << 20, BIG, None) == status
        assert L.svp_pages_compact(pages(**bad), caches(), 1, 2, 128, None, 1 << 20, BIG, None) == status
    sizes = []
    for count in (0, 1, 100, 1 << 20):
        assert L.svp_pages_workspace_size(pages(num_pages=count), ctypes.byref(nb)) == OK
        sizes.append(nb.value)
    assert sizes == sorted(sizes) and sizes[0] >= 256 and sizes[-1] >= 8 << 20


def test_refusals(L):
    nb = ctypes.c_size_t(0)
    L.svp_pages_workspace_size(pages(), ctypes.byref(nb))
    resize = lambda p=pages(), length=16, ws=1 << 20, wsb=BIG: L.svp_pages_resize(p, length, ws, wsb, None)
    assert resize(length=None) == INV and resize(ws=(1 << 20) + 4) == INV
    assert resize(p=None) == INV and resize(ws=None) == WSP and resize(wsb=nb.value - 1) == WSP
    for name in ("block_table", "used", "refs"):
        assert resize(p=pages(**{name: None})) == INV
    assert resize(p=pages(n=0), length=None) == OK
    fork = lambda p=pages(), ca=caches(), count=1, hkv=2, d=128, src=16, dst=16, length=16, forks=1, ws=1 << 20, wsb=BIG: \
        L.svp_pages_fork(p, ca, count, hkv, d, src, dst, length, forks, ws, wsb, None)
    assert fork(src=None) == INV and fork(dst=None) == INV and fork(length=None) == INV and fork(forks=-1) == INV
    assert fork(forks=1025) == UNS and fork(ws=None) == WSP and fork(wsb=nb.value - 1) == WSP and fork(p=None) == INV
    assert fork(forks=0) == OK and fork(p=pages(n=0)) == OK and fork(forks=0, ca=None, count=0) == OK
    compact = lambda p=pages(), ca=caches(), count=1, hkv=2, d=128, ws=1 << 20, wsb=BIG: \
        L.svp_pages_compact(p, ca, count, hkv, d, None, ws, wsb, None)
    assert compact(p=None) == INV and compact(p=pages(refs=None)) == INV and compact(p=pages(used=None)) == INV
    assert compact(ws=None) == WSP and compact(wsb=nb.value - 1) == WSP
    for call in (fork, compact):
        assert call(ca=None) == INV and call(count=-1) == INV and call(count=65, ca=caches(65)) == UNS
        assert call(hkv=0) == INV and call(hkv=5000) == UNS and call(d=96) == UNS
        for bad in (dict(page_size=32), dict(num_pages=99), dict(k=None), dict(stride_tok=64), dict(k=(1 << 20) + 8)):
            assert call(ca=caches(1, **bad)) == INV
        for bad in (dict(dtype=svp.SVP_F32), dict(stride_page=2 * 16 * 128 + 8), dict(stride_head=16 * 128 + 8)):
            assert call(ca=caches(2, **bad), count=2) == INV       # unlike the first
        assert call(ca=caches(1, dtype=svp.SVP_E4M3)) == INV       # no exponent bytes


def test_binding_refuses_cpu_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        svp.make_pages(z.view(2, 2), z[:2], z, page_size=16)
