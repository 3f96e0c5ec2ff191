"""Rotary positions on the host (no GPU): the frequency tables against their formulas, and every
refusal before any CUDA call."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_verification_packed_gb300 as svp
from speculative_decoding_verification_packed_gb300 import build as svp_build

OK, INV, UNS, WSP = svp.SVP_OK, svp.SVP_EINVAL, svp.SVP_EUNSUPPORTED, svp.SVP_EWORKSPACE
BIG = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def L():
    svp_build.build()
    return svp.lib()


def turns(table):
    return [(int(x) & (2 ** 64 - 1)) / 2.0 ** 64 for x in table.tolist()]


def expect(rot, base, way, factor, original, slow=1.0, fast=32.0):
    """Radians a position of each pair, from the formulas."""
    out = []
    for t in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if way == "ntk" and rot > 2 else base
        f = b ** (-2 * t / rot)
        if way == "linear":
            f /= factor
        if way == "yarn":
            lo = max(math.floor(rot * math.log(original / (fast * 2 * math.pi)) / (2 * math.log(base))), 0)
            hi = min(math.ceil(rot * math.log(original / (slow * 2 * math.pi)) / (2 * math.log(base))), rot - 1)
            ramp = min(max((t - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            f = f * (1 - ramp) + f / factor * ramp
        out.append(f)
    return out


@pytest.mark.parametrize("rot", [2, 16, 18, 64, 128, 256])
@pytest.mark.parametrize("way,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 8.0), ("yarn", 1.0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(rot, way, factor, base):
    got = turns(svp.rope_frequencies(rot, base=base, scaling=way, factor=factor, original=4096, device="cpu"))
    for a, b in zip(got, expect(rot, base, way, factor, 4096)):
        # a power, a product and a quotient in 64 bits: a few 2^-53 of the value, times ln of the base; and the
        # table's unit, 2^-64 of a turn = 2 pi 2^-64 < 2^-61 radians, below which it is cut off
        assert abs(a * 2 * math.pi - b) <= 64 * 2.0 ** -53 * b + 2.0 ** -61


def test_yarn_keeps_fast_pairs_and_stretches_slow_ones():
    plain = turns(svp.rope_frequencies(128, device="cpu"))
    y = turns(svp.rope_frequencies(128, scaling="yarn", factor=16.0, original=4096, device="cpu"))
    for a, b in zip(plain, y):
        if a * 4096 > 64:
            assert a == b
        # (both tables are cut off at 2^-64, and 64-bit arithmetic is off by a few 2^-53)
        if a * 4096 < 0.5:
            assert abs(b - a / 16) <= 1e-15 * a + 2.0 ** -63
        assert a / 16 * (1 - 1e-15) - 2.0 ** -63 <= b <= a + 2.0 ** -63


def test_frequency_refusals(L):
    out = (ctypes.c_uint64 * 64)()
    f = lambda rot=16, base=1e4, way=0, factor=1.0, original=4096, slow=1.0, fast=32.0, o=out: \
        L.svp_rope_frequencies(rot, base, way, factor, original, slow, fast, o)
    assert f() == OK
    assert f(rot=0) == INV and f(rot=15) == INV and f(rot=-2) == INV and f(base=1.0) == INV and f(base=0.5) == INV
    assert f(base=float("nan")) == INV and f(base=float("inf")) == INV and f(factor=0.0) == INV and f(factor=-1.0) == INV
    assert f(factor=float("inf")) == INV and f(o=None) == INV and f(way=4) == UNS and f(way=-1) == UNS
    assert f(way=3, original=0) == INV and f(way=3, slow=0.0) == INV and f(way=3, slow=32.0) == INV
    assert f(way=3, fast=float("inf")) == INV and f(way=2, original=0, slow=0.0) == OK
    with pytest.raises(ValueError):
        svp.rope_frequencies(16, scaling="other", device="cpu")


def rotary(**kw):
    r = svp.svp_rotary(16, 64, 0, 1.0)
    for name, x in kw.items():
        setattr(r, name, x)
    return ctypes.byref(r)


BAD_ROTARY = [dict(rot=0), dict(rot=63), dict(rot=130), dict(rot=-2), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(interleaved=2), dict(interleaved=-1), dict(freq=None)]


def test_rope_refusals(L):
    f = lambda q=16, qs=512, k=16, ks=256, dtype=1, rot=rotary(), pos=None, ctx=16, cu=16, n=1, m=4, hq=4, hkv=2, d=128, \
        qo=32, qos=512, ko=32, kos=256, ws=16, wsb=BIG: \
        L.svp_rope(q, qs, k, ks, dtype, rot, pos, ctx, cu, n, m, hq, hkv, d, qo, qos, ko, kos, ws, wsb, None)
    for bad in BAD_ROTARY:
        assert f(rot=rotary(**bad)) == INV
    assert f(rot=None) == INV and f(n=-1) == INV and f(m=-1) == INV and f(hq=0) == INV and f(hkv=-1) == INV
    assert f(q=None) == INV and f(qo=None) == INV and f(k=None) == INV and f(ko=None) == INV
    assert f(qs=511) == INV and f(qs=516) == INV and f(qos=510) == INV and f(ks=255) == INV and f(kos=260) == INV
    assert f(q=8) == INV and f(qo=40) == INV and f(k=24) == INV and f(ko=8) == INV
    assert f(q=16, qo=16, qos=520) == INV and f(k=16, ko=16, ks=264) == INV        # in place, other strides
    assert f(ctx=None) == INV and f(cu=None) == INV and f(cu=None, pos=16) == INV
    assert f(d=96) == UNS and f(dtype=2) == UNS and f(dtype=7) == UNS
    assert f(ws=None) == WSP and f(wsb=255) == WSP
    assert f(n=0) == OK and f(m=0) == OK and f(q=None, qo=None, k=None, ko=None) == OK
    assert f(q=None, qo=None, hq=0, n=0) == OK and f(k=None, ko=None, hkv=0, n=0) == OK


def test_rope_cache_write_refusals(L):
    c = svp.svp_cache()
    c.k = c.v = c.k_exp = c.v_exp = c.block_table = 1 << 20
    c.max_pages, c.page_size, c.num_pages = 8, 16, 100
    c.stride_page, c.stride_head, c.stride_tok, c.dtype = 2 * 16 * 128, 16 * 128, 128, svp.SVP_BF16
    f = lambda q=16, qs=512, k=16, v=16, ks=256, dtype=1, rot=rotary(), ca=ctypes.byref(c), ctx=16, cu=16, n=1, m=4, hq=4, \
        hkv=2, d=128, qo=32, qos=512, ws=16, wsb=BIG: \
        L.svp_rope_cache_write(q, qs, k, v, ks, dtype, rot, ca, None, ctx, cu, None, n, m, hq, hkv, d, qo, qos, ws, wsb, None)
    for bad in BAD_ROTARY:
        assert f(rot=rotary(**bad)) == INV
    assert f(rot=None) == INV and f(ca=None) == INV and f(n=-1) == INV and f(m=-1) == INV and f(hq=0) == INV and f(hkv=0) == INV
    assert f(q=None) == INV and f(qo=None) == INV and f(k=None) == INV and f(v=None) == INV and f(v=8) == INV and f(k=24) == INV
    assert f(qs=511) == INV and f(qos=516) == INV and f(ks=255) == INV and f(q=16, qo=16, qos=520) == INV
    assert f(ctx=None) == INV and f(cu=None) == INV
    assert f(d=96) == UNS and f(dtype=2) == UNS
    assert f(ws=None) == WSP and f(wsb=64) == WSP
    assert f(n=0) == OK and f(m=0) == OK and f(q=None, qo=None, n=0) == OK
    c.page_size = 48
    assert f() == UNS


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    freq = svp.rope_frequencies(64, device="cpu")
    with pytest.raises(ValueError):
        svp.rope(x, x, None, torch.zeros(2, dtype=torch.int32), freq=freq, pos=torch.zeros(2, dtype=torch.int32))
