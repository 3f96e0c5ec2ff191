"""Alignment of the attention's workspaces, on the host (no GPU): partial results are stored 32 bytes at a time, so a
workspace on less than a 32-byte boundary is refused before any CUDA call."""
import ctypes

import pytest

import speculative_decoding_verification_packed_gb300 as svp
from speculative_decoding_verification_packed_gb300 import build as svp_build
from test_cache_abi import cache

BASE, BIG = 1 << 20, 1 << 40


@pytest.fixture(scope="module", autouse=True)
def L():
    svp_build.build()
    return svp.lib()


@pytest.mark.parametrize("kind", [svp.SVP_BF16, svp.SVP_E4M3])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,rows", [(2, 1), (4, 4), (32, 64)])
@pytest.mark.parametrize("off", [1, 4, 8, 16, 24, 48, 16 + 256])
def test_a_workspace_between_32_byte_boundaries_is_refused(L, kind, d, hq, rows, off):
    c = cache(dtype=kind, stride_page=2 * 16 * d, stride_head=16 * d, stride_tok=d)
    h = ctypes.byref(svp.svp_heads(hq, 2, d, 0.0))
    ca = ctypes.byref(c)
    assert L.svp_chunk_attn(16, hq * d, ca, 16, 16, 1, rows, rows, h, svp.SVP_BF16, 16, None, BASE + off, BIG,
                            None) == svp.SVP_EINVAL
    for groups in (0, 1):
        assert L.svp_prefix_attn(16, hq * d, ca, 16, 16, 1, rows, rows, 16, 16, groups, h, svp.SVP_BF16, 16, None,
                                 BASE + off, BIG, None) == svp.SVP_EINVAL
    # what does nothing does not look at it
    assert L.svp_chunk_attn(16, hq * d, ca, 16, 16, 0, rows, rows, h, svp.SVP_BF16, 16, None, BASE + off, BIG,
                            None) == svp.SVP_OK
    assert L.svp_prefix_attn(16, hq * d, ca, 16, 16, 1, 0, rows, 16, 16, 1, h, svp.SVP_BF16, 16, None, BASE + off, BIG,
                             None) == svp.SVP_OK
