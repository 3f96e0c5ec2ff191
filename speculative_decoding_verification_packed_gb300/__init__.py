"""Packed speculative-verification attention and margin/accept for GB300 (sm_103a).

A thin Python binding over the C ABI of ``include/svp.h`` (``libsvp.so``, built in-tree
by ``build.py``).  The functions here only marshal torch CUDA tensors into pointers,
sizes and the current stream; every step of the computation runs in the library's
CUDA kernels.  There is no CPU fallback: if the library is missing or the tensors are
not on a CUDA device, the call raises.

Entry points (same names as the C ABI, without the ``svp_`` prefix):
  verify_attn_packed   attention of packed candidate rows over their request's KV
                       context and their own earlier candidates (contiguous or paged KV,
                       GQA); ``tile_mode`` selects the contrast tiles
  prefill_attn         wide-tile causal prefill attention
  draft_margin         per-row top-1 index/value, top-2 value and fp32 margin
  greedy_accept        longest matching draft prefix and successor token per request
  margin_accept        draft_margin over packed target rows fused with greedy_accept
  cache_write          new key / value rows (or their accepted prefixes) into the pages of a
                       cache in fp32, bf16 or 8 bits with an exponent per row (make_cache)
  cache_read           cached positions back to contiguous rows
  chunk_attn           attention of decode tokens, candidate blocks and prompt chunks whose
                       keys and values are in the cache already
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvp.so")

SVP_OK, SVP_EINVAL, SVP_EUNSUPPORTED, SVP_EWORKSPACE, SVP_ECUDA = 0, 1, 2, 3, 4
SVP_F32, SVP_BF16, SVP_E4M3 = 0, 1, 2
TILE_AUTO, TILE_SHORT, TILE_FIXED128, TILE_WIDE, TILE_SHORT_UNPACKED = 0, 1, 2, 3, 4
DEV_BAD_SLOTS, DEV_BAD_CONTEXT, DEV_TIMEOUT, DEV_WORKSPACE = 0x1, 0x2, 0x4, 0x8


class SvpError(RuntimeError):
    """A library call returned a non-OK status."""

    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class svp_heads(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class svp_kv(ctypes.Structure):
    _fields_ = [("paged", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("cu_ctx", ctypes.c_void_p), ("total_tokens", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("stride_page", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("stride_tok", ctypes.c_int64)]


class svp_gather_field(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("src_rows", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64), ("dst", ctypes.c_void_p)]


class svp_cache(ctypes.Structure):
    """A paged cache for cache_write / cache_read / chunk_attn; see make_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("stride_page", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("stride_tok", ctypes.c_int64),
                ("dtype", ctypes.c_int)]


GATHER_MAX_FIELDS = 8

_lib = None

_SIGS = {
    "svp_version": (ctypes.c_int32, []),
    "svp_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "svp_workspace_init": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_read_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.POINTER(ctypes.c_int32)]),
    "svp_verify_attn_workspace_size": (ctypes.c_int, [
        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(svp_heads), ctypes.c_int,
        ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "svp_verify_attn_packed": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(svp_kv),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
        ctypes.POINTER(svp_heads), ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_verify_attn_packed_ex": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(svp_kv),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
        ctypes.POINTER(svp_heads), ctypes.c_int, ctypes.c_int32, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_prefill_attn_workspace_size": (ctypes.c_int, [
        ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(svp_heads), ctypes.c_int,
        ctypes.POINTER(ctypes.c_size_t)]),
    "svp_prefill_attn": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.POINTER(svp_heads), ctypes.c_int,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_draft_margin_workspace_size": (ctypes.c_int, [
        ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "svp_draft_margin": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "svp_greedy_accept": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "svp_margin_accept_workspace_size": (ctypes.c_int, [
        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "svp_dvl_allocate_pack": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "svp_gather_rows": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int32,
        ctypes.c_void_p, ctypes.c_void_p]),
    "svp_gather_rows_multi": (ctypes.c_int, [
        ctypes.POINTER(svp_gather_field), ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
        ctypes.c_void_p]),
    "svp_stochastic_accept_workspace_size": (ctypes.c_int, [
        ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "svp_stochastic_accept": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
    "svp_draft_features_workspace_size": (ctypes.c_int, [
        ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "svp_draft_features": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_act_truncate": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
        ctypes.c_void_p, ctypes.c_void_p]),
    "svp_cache_write": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER(svp_cache),
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_cache_read": (ctypes.c_int, [
        ctypes.POINTER(svp_cache), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
        ctypes.c_int32, ctypes.c_int32, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "svp_chunk_attn_workspace_size": (ctypes.c_int, [
        ctypes.POINTER(svp_heads), ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]),
    "svp_chunk_attn": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(svp_cache), ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(svp_heads),
        ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
        ctypes.c_void_p]),
    "svp_margin_accept": (ctypes.c_int, [
        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
        ctypes.c_size_t, ctypes.c_void_p]),
}


def lib() -> ctypes.CDLL:
    """The loaded libsvp.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libsvp.so is not built ({LIB_PATH}); run "
                "`python -m speculative_decoding_verification_packed_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().svp_status_string(int(status)).decode()
    except Exception:  # library missing: still produce a message
        return f"status {status}"


def _check(status: int, what: str) -> None:
    if status != SVP_OK:
        raise SvpError(status, what)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SVP_BF16
    if t.dtype == torch.float32:
        return SVP_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _dev(t: Optional[torch.Tensor], name: str, dtype=None) -> int:
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class Workspace:
    """Device scratch for one entry point, zeroed once at creation (svp_workspace_init).

    The clear is enqueued on ``stream`` (default: the current stream).  A call on another
    stream must be ordered after it (the same stream, a synchronize, or an event): torch's
    side streams do not wait for the default stream."""

    def __init__(self, nbytes: int, device=None, stream=None, zeroed: Optional[int] = None):
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        # (zeroed: the leading bytes that the entry point wants zeroed; None for all of them)
        if zeroed != 0:
            _check(lib().svp_workspace_init(self.ptr, self.nbytes if zeroed is None else zeroed, _stream(stream)),
                   "svp_workspace_init")

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def read_status(self, stream=None) -> int:
        """Device status bits since the last read (synchronises the stream)."""
        v = ctypes.c_int32(0)
        _check(lib().svp_read_status(self.ptr, _stream(stream), ctypes.byref(v)),
               "svp_read_status")
        return int(v.value)


_ws_cache: dict = {}


def _workspace(key, nbytes: int, device, stream) -> Workspace:
    ws = _ws_cache.get((key, device))
    if ws is None or ws.nbytes < nbytes:
        ws = Workspace(nbytes, device, stream)
        _ws_cache[(key, device)] = ws
    return ws


def _heads(hq: int, hkv: int, d: int, scale: float) -> svp_heads:
    return svp_heads(int(hq), int(hkv), int(d), float(scale))


# ----------------------------------------------------------------- attention
def verify_attn_workspace_size(n: int, m_cap: int, w: int, hq: int, hkv: int, d: int,
                               dtype=torch.bfloat16, tile_mode: int = TILE_AUTO) -> int:
    out = ctypes.c_size_t(0)
    code = SVP_BF16 if dtype == torch.bfloat16 else SVP_F32
    h = _heads(hq, hkv, d, 0.0)
    _check(lib().svp_verify_attn_workspace_size(n, m_cap, w, ctypes.byref(h), code, tile_mode,
                                                ctypes.byref(out)),
           "svp_verify_attn_workspace_size")
    return int(out.value)


def make_kv(*, k_ctx=None, v_ctx=None, cu_ctx=None, k_cache=None, v_cache=None,
            block_table=None, page_size: int = 16) -> svp_kv:
    """svp_kv for contiguous (k_ctx, v_ctx, cu_ctx) or paged (k_cache, v_cache,
    block_table) committed context; None for both means no context."""
    kv = svp_kv()
    if k_cache is not None:
        if k_cache.stride() != v_cache.stride() or k_cache.stride(-1) != 1:
            raise ValueError("k_cache and v_cache need identical strides, last dim contiguous")
        kv.paged = 1
        kv.k = k_cache.data_ptr()
        kv.v = v_cache.data_ptr()
        _dev(block_table, "block_table", torch.int32)
        kv.block_table = block_table.data_ptr()
        kv.max_pages = block_table.shape[1]
        kv.page_size = page_size
        kv.num_pages = k_cache.shape[0]
        s = k_cache.stride()
        kv.stride_page, kv.stride_head, kv.stride_tok = s[0], s[1], s[2]
        if k_cache.device.type != "cuda" or v_cache.device.type != "cuda":
            raise ValueError("KV cache must be on a CUDA device")
    elif k_ctx is not None:
        kv.paged = 0
        kv.k = _dev(k_ctx, "k_ctx")
        kv.v = _dev(v_ctx, "v_ctx")
        kv.cu_ctx = _dev(cu_ctx, "cu_ctx", torch.int64)
        kv.total_tokens = k_ctx.shape[0]
    return kv


def verify_attn_packed(q, k_new, v_new, ctx_len, cu_slots, *, w: int, hkv: Optional[int] = None,
                       kv: Optional[svp_kv] = None, out=None, lse=None, want_lse: bool = True,
                       scale: float = 0.0, tile_mode: int = TILE_AUTO, ws: Optional[Workspace] = None,
                       stream=None, **kv_tensors):
    """Verification attention; returns (out [m_cap, hq, d], lse [m_cap, hq] or None).

    q [m_cap, hq, d]; k_new, v_new [m_cap, hkv, d]; ctx_len [n] int32; cu_slots [n+1]
    int32; context via ``kv`` (see make_kv) or the make_kv keyword tensors.
    """
    m_cap, hq, d = q.shape
    hkv = hkv if hkv is not None else k_new.shape[1]
    n = cu_slots.shape[0] - 1
    code = _dtype_code(q)
    if kv is None:
        kv = make_kv(**kv_tensors)
    if out is None:
        out = torch.full_like(q, float("nan"))
    if lse is None and want_lse:
        lse = torch.full((m_cap, hq), float("nan"), dtype=torch.float32, device=q.device)
    nbytes = verify_attn_workspace_size(n, m_cap, w, hq, hkv, d, q.dtype, tile_mode)
    if ws is None:
        ws = _workspace(("verify", tile_mode, code, d), nbytes, q.device, stream)
    h = _heads(hq, hkv, d, scale)
    _check(lib().svp_verify_attn_packed_ex(
        _dev(q, "q"), _dev(k_new, "k_new"), _dev(v_new, "v_new"), ctypes.byref(kv),
        _dev(ctx_len, "ctx_len", torch.int32), _dev(cu_slots, "cu_slots", torch.int32),
        n, m_cap, int(w), ctypes.byref(h), code, int(tile_mode), _dev(out, "out"),
        _dev(lse, "lse", torch.float32), ws.ptr, ws.nbytes, _stream(stream)),
        "svp_verify_attn_packed")
    return out, lse


def prefill_attn_workspace_size(n: int, max_s: int, hq: int, hkv: int, d: int) -> int:
    out = ctypes.c_size_t(0)
    h = _heads(hq, hkv, d, 0.0)
    _check(lib().svp_prefill_attn_workspace_size(n, max_s, ctypes.byref(h), SVP_BF16,
                                                 ctypes.byref(out)),
           "svp_prefill_attn_workspace_size")
    return int(out.value)


def prefill_attn(q, k, v, cu_seqlens, *, max_s: int, out=None, lse=None, want_lse=True,
                 scale: float = 0.0, ws: Optional[Workspace] = None, stream=None):
    """Causal prefill attention of packed sequences; returns (out, lse)."""
    total_s, hq, d = q.shape
    hkv = k.shape[1]
    n = cu_seqlens.shape[0] - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((total_s, hq), dtype=torch.float32, device=q.device)
    nbytes = prefill_attn_workspace_size(n, max_s, hq, hkv, d)
    if ws is None:
        ws = _workspace(("prefill", d), nbytes, q.device, stream)
    h = _heads(hq, hkv, d, scale)
    _check(lib().svp_prefill_attn(
        _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(cu_seqlens, "cu_seqlens", torch.int32),
        n, int(max_s), int(total_s), 1, ctypes.byref(h), _dtype_code(q), _dev(out, "out"),
        _dev(lse, "lse", torch.float32), ws.ptr, ws.nbytes, _stream(stream)),
        "svp_prefill_attn")
    return out, lse


# ----------------------------------------------------------------- margin / accept
def draft_margin_workspace_size(rows: int, vocab: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().svp_draft_margin_workspace_size(rows, vocab, ctypes.byref(out)),
           "svp_draft_margin_workspace_size")
    return int(out.value)


def draft_margin(logits, *, vocab: Optional[int] = None, ws: Optional[Workspace] = None,
                 outs=None, stream=None):
    """(top1_idx int32, top1 f32, top2 f32, margin f32) per row of logits [rows, V]."""
    rows, stride = logits.shape
    vocab = stride if vocab is None else vocab
    dev = logits.device
    if outs is None:
        outs = (torch.empty(rows, dtype=torch.int32, device=dev),
                torch.empty(rows, dtype=torch.float32, device=dev),
                torch.empty(rows, dtype=torch.float32, device=dev),
                torch.empty(rows, dtype=torch.float32, device=dev))
    idx, t1, t2, mg = outs
    if ws is None:
        ws = _workspace(("margin",), draft_margin_workspace_size(rows, vocab), dev, stream)
    _check(lib().svp_draft_margin(
        _dev(logits, "logits"), stride, rows, vocab, _dtype_code(logits),
        _dev(idx, "top1_idx", torch.int32), _dev(t1, "top1", torch.float32),
        _dev(t2, "top2", torch.float32), _dev(mg, "margin", torch.float32),
        ws.ptr, ws.nbytes, _stream(stream)), "svp_draft_margin")
    return outs


def greedy_accept(target_argmax, tokens, cu_slots, *, outs=None, stream=None):
    """(accept_len [n] int32, next_token [n] int32)."""
    n = cu_slots.shape[0] - 1
    m_cap = tokens.shape[0]
    dev = tokens.device
    if outs is None:
        outs = (torch.empty(n, dtype=torch.int32, device=dev),
                torch.empty(n, dtype=torch.int32, device=dev))
    acc, nxt = outs
    _check(lib().svp_greedy_accept(
        _dev(target_argmax, "target_argmax", torch.int32), _dev(tokens, "tokens", torch.int32),
        _dev(cu_slots, "cu_slots", torch.int32), n, m_cap, _dev(acc, "accept_len", torch.int32),
        _dev(nxt, "next_token", torch.int32), _stream(stream)), "svp_greedy_accept")
    return outs


def margin_accept_workspace_size(n: int, m_cap: int, vocab: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().svp_margin_accept_workspace_size(n, m_cap, vocab, ctypes.byref(out)),
           "svp_margin_accept_workspace_size")
    return int(out.value)


def margin_accept(logits, tokens, cu_slots, *, vocab: Optional[int] = None,
                  ws: Optional[Workspace] = None, outs=None, stream=None):
    """Fused row margin over packed target logits [m_cap, V] + greedy acceptance.

    Returns (top1_idx, top1, top2, margin) per row and (accept_len, next_token) per
    request.  Rows >= cu_slots[n] are neither read nor written."""
    m_cap, stride = logits.shape
    vocab = stride if vocab is None else vocab
    n = cu_slots.shape[0] - 1
    dev = logits.device
    if outs is None:
        outs = (torch.full((m_cap,), -1, dtype=torch.int32, device=dev),
                torch.full((m_cap,), float("nan"), dtype=torch.float32, device=dev),
                torch.full((m_cap,), float("nan"), dtype=torch.float32, device=dev),
                torch.full((m_cap,), float("nan"), dtype=torch.float32, device=dev),
                torch.empty(n, dtype=torch.int32, device=dev),
                torch.empty(n, dtype=torch.int32, device=dev))
    idx, t1, t2, mg, acc, nxt = outs
    if ws is None:
        ws = _workspace(("margin_accept",), margin_accept_workspace_size(n, m_cap, vocab), dev,
                        stream)
    _check(lib().svp_margin_accept(
        _dev(logits, "logits"), stride, m_cap, vocab, _dtype_code(logits),
        _dev(tokens, "tokens", torch.int32), _dev(cu_slots, "cu_slots", torch.int32), n,
        _dev(idx, "top1_idx", torch.int32), _dev(t1, "top1", torch.float32),
        _dev(t2, "top2", torch.float32), _dev(mg, "margin", torch.float32),
        _dev(acc, "accept_len", torch.int32), _dev(nxt, "next_token", torch.int32),
        ws.ptr, ws.nbytes, _stream(stream)), "svp_margin_accept")
    return outs


def dvl_allocate_pack(scores, *, n_live=None, budget_per_req: int = 8, m_cap: Optional[int] = None,
                      tokens=None, positions=None, kv_refs=None, fill_token: int = 0,
                      fill_pos: int = 0, fill_ref: int = -1, ws: Optional[Workspace] = None,
                      stream=None) -> Dict[str, torch.Tensor]:
    """DVL budget allocator + flat-buffer packer (svp_dvl_allocate_pack).

    scores [n_bs, w-1] fp32 acceptance scores; n_live: device int32 scalar tensor or None
    (all live); tokens / positions / kv_refs [n_bs, w] int32 or None.  Returns k_init,
    k, cu_slots, n_adjust and the packed fields that were given.
    """
    if scores.dim() != 2:
        raise SvpError("scores must be [n_bs, w-1]")
    n_bs, wm1 = scores.shape
    w = wm1 + 1
    dev = scores.device
    if m_cap is None:
        m_cap = w * n_bs
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(k_init=torch.empty(n_bs, **i32), k=torch.empty(n_bs, **i32),
               cu_slots=torch.empty(n_bs + 1, **i32), n_adjust=torch.empty(1, **i32))
    for name, f in (("tokens", tokens), ("positions", positions), ("kv_refs", kv_refs)):
        if f is not None:
            if tuple(f.shape) != (n_bs, w):
                raise SvpError(f"{name} must be [n_bs, w]")
            out[name] = torch.empty(m_cap, **i32)
    if ws is None:
        ws = _workspace(("dvl",), 256, dev, stream)
    st = lib().svp_dvl_allocate_pack(
        _dev(scores, "scores", torch.float32), n_bs, w,
        _dev(n_live, "n_live", torch.int32) if n_live is not None else None, budget_per_req,
        _dev(tokens, "tokens", torch.int32) if tokens is not None else None,
        _dev(positions, "positions", torch.int32) if positions is not None else None,
        _dev(kv_refs, "kv_refs", torch.int32) if kv_refs is not None else None,
        m_cap, fill_token, fill_pos, fill_ref,
        out["k_init"].data_ptr(), out["k"].data_ptr(), out["cu_slots"].data_ptr(),
        out["tokens"].data_ptr() if "tokens" in out else None,
        out["positions"].data_ptr() if "positions" in out else None,
        out["kv_refs"].data_ptr() if "kv_refs" in out else None,
        out["n_adjust"].data_ptr(), ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "svp_dvl_allocate_pack")
    out["ws"] = ws
    return out


def gather_rows_multi(srcs, idx, *, outs=None, stream=None):
    """svp_gather_rows_multi: the packed copy of several wide per-row fields sharing the row
    map idx, in one launch; returns the list of outputs."""
    rows = idx.shape[0]
    if not 1 <= len(srcs) <= GATHER_MAX_FIELDS:
        raise ValueError(f"gather_rows_multi takes 1..{GATHER_MAX_FIELDS} fields")
    if outs is None:
        outs = [torch.empty((rows,) + tuple(s.shape[1:]), dtype=s.dtype, device=s.device) for s in srcs]
    fields = (svp_gather_field * len(srcs))()
    for f, (s, o) in enumerate(zip(srcs, outs)):
        rb = s[0].numel() * s.element_size() if s.shape[0] else o[0].numel() * o.element_size()
        fields[f] = svp_gather_field(_dev(s, f"srcs[{f}]"), s.shape[0], rb, _dev(o, f"outs[{f}]"))
    _check(lib().svp_gather_rows_multi(fields, len(srcs), _dev(idx, "idx", torch.int32), rows,
                                       _stream(stream)), "svp_gather_rows_multi")
    return outs


def gather_rows(src, idx, *, out=None, stream=None):
    """Packed copy of a wide per-row field (svp_gather_rows): out[r] = src[idx[r]] for
    in-range ids, zeros otherwise.  src [src_rows, ...] contiguous; idx [rows] int32."""
    rows = idx.shape[0]
    if out is None:
        out = torch.empty((rows,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    row_bytes = src[0].numel() * src.element_size() if src.shape[0] else out[0].numel() * out.element_size()
    _check(lib().svp_gather_rows(_dev(src, "src"), src.shape[0], row_bytes,
                                 _dev(idx, "idx", torch.int32), rows, _dev(out, "out"),
                                 _stream(stream)), "svp_gather_rows")
    return out


def stochastic_accept_workspace_size(m_cap: int, vocab: int) -> int:
    nb = ctypes.c_size_t(0)
    _check(lib().svp_stochastic_accept_workspace_size(m_cap, vocab, ctypes.byref(nb)),
           "svp_stochastic_accept_workspace_size")
    return int(nb.value)


def stochastic_accept(logits, tokens, cu_slots, u_accept, u_next, *, temperature: float,
                      vocab: Optional[int] = None, ws: Optional[Workspace] = None, outs=None,
                      stream=None):
    """Stochastic prefix verifier (svp_stochastic_accept); returns (accept_len [n],
    next_token [n], p_draft [m_cap])."""
    m_cap, stride = logits.shape
    vocab = stride if vocab is None else vocab
    n = cu_slots.shape[0] - 1
    dev = logits.device
    if outs is None:
        outs = (torch.empty(n, dtype=torch.int32, device=dev),
                torch.empty(n, dtype=torch.int32, device=dev),
                torch.full((m_cap,), float("nan"), dtype=torch.float32, device=dev))
    acc, nxt, pd = outs
    if ws is None:
        ws = _workspace(("stochastic",), stochastic_accept_workspace_size(m_cap, vocab), dev, stream)
    _check(lib().svp_stochastic_accept(
        _dev(logits, "logits"), stride, m_cap, vocab, _dtype_code(logits),
        _dev(tokens, "tokens", torch.int32), _dev(cu_slots, "cu_slots", torch.int32), n,
        float(temperature), _dev(u_accept, "u_accept", torch.float32),
        _dev(u_next, "u_next", torch.float32), _dev(acc, "accept_len", torch.int32),
        _dev(nxt, "next_token", torch.int32), _dev(pd, "p_draft", torch.float32) if pd is not None else None,
        ws.ptr, ws.nbytes, _stream(stream)), "svp_stochastic_accept")
    return outs


def draft_features_workspace_size(rows: int, vocab: int) -> int:
    nb = ctypes.c_size_t(0)
    _check(lib().svp_draft_features_workspace_size(rows, vocab, ctypes.byref(nb)),
           "svp_draft_features_workspace_size")
    return int(nb.value)


def draft_features(logits, *, vocab: Optional[int] = None, out=None, ws: Optional[Workspace] = None,
                   stream=None):
    """[rows, 18] fp32 draft-signal features of every logit row (svp_draft_features)."""
    rows, stride = logits.shape
    vocab = stride if vocab is None else vocab
    if out is None:
        out = torch.empty(rows, 18, dtype=torch.float32, device=logits.device)
    if ws is None:
        ws = _workspace(("features",), draft_features_workspace_size(rows, vocab), logits.device, stream)
    _check(lib().svp_draft_features(_dev(logits, "logits"), stride, rows, vocab, _dtype_code(logits),
                                    _dev(out, "features", torch.float32), ws.ptr, ws.nbytes,
                                    _stream(stream)), "svp_draft_features")
    return out


def act_truncate(margins, *, n: int, w: int, threshold: float, stride: int = 1, out=None, stream=None):
    """k [n] int32 after ACT truncation of margins laid out per request and position."""
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=margins.device)
    _check(lib().svp_act_truncate(_dev(margins, "margins", torch.float32), stride, n, w,
                                  float(threshold), _dev(out, "k", torch.int32), _stream(stream)),
           "svp_act_truncate")
    return out


# ----------------------------------------------------------------- paged cache
_CACHE_DTYPES = {torch.float32: SVP_F32, torch.bfloat16: SVP_BF16, torch.float8_e4m3fn: SVP_E4M3}


def make_cache(k_cache, v_cache, block_table, *, k_exp=None, v_exp=None) -> svp_cache:
    """svp_cache over page pools k_cache / v_cache [pages, hkv, page_size, d] (fp32, bf16 or
    float8_e4m3fn; any strides with the last dim contiguous, so pools laid out [pages,
    page_size, hkv, d] are given as their transpose(1, 2)) and block_table [n, max_pages] int32.
    float8_e4m3fn pools need k_exp / v_exp [pages, hkv, page_size] uint8: an element is its
    code times 2^(byte - 127).  The struct keeps the tensors alive."""
    for name, x in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
        if x.dim() != 4 or x.dtype not in _CACHE_DTYPES:
            raise TypeError(f"{name} must be [pages, hkv, page_size, d] in fp32, bf16 or float8_e4m3fn")
    if (k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype
            or k_cache.stride() != v_cache.stride() or k_cache.stride(-1) != 1):
        raise ValueError("k_cache and v_cache need one shape, type and strides, last dim contiguous")
    c = svp_cache()
    c.k, c.v, c.dtype = k_cache.data_ptr(), v_cache.data_ptr(), _CACHE_DTYPES[k_cache.dtype]
    c.num_pages, c.hkv, c.page_size, c.d = k_cache.shape
    c.stride_page, c.stride_head, c.stride_tok = k_cache.stride()[:3]
    c.block_table = _dev(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [n, max_pages]")
    c.max_n, c.max_pages = block_table.shape
    if c.dtype == SVP_E4M3:
        for name, x in (("k_exp", k_exp), ("v_exp", v_exp)):
            if x is None or tuple(x.shape) != tuple(k_cache.shape[:3]):
                raise ValueError(f"an 8-bit cache needs {name} [pages, hkv, page_size]")
        c.k_exp, c.v_exp = _dev(k_exp, "k_exp", torch.uint8), _dev(v_exp, "v_exp", torch.uint8)
    elif k_exp is not None or v_exp is not None:
        raise ValueError("exponent bytes belong to float8_e4m3fn pools")
    c.device, c.index, c.ws = k_cache.device, k_cache.device.index, None
    c.keep = (k_cache, v_cache, k_exp, v_exp, block_table)
    for x in c.keep:
        if x is not None and x.device != c.device:
            raise ValueError("the cache's tensors must be on one device")
    return c


# These three run once a decode step and layer, so their checks cost little: plain attribute reads, and
# the current stream's raw handle.
def _rows(t, name: str, heads: int, cache: svp_cache) -> int:
    """Row stride of rows [m, heads, d] whose heads and elements are contiguous."""
    d = cache.d
    m, h, e = t.shape
    if h != heads or e != d:
        raise ValueError(f"{name} must be [rows, {heads}, {d}]")
    s0, s1, s2 = t.stride()
    if t.get_device() != cache.index or s2 != 1 or (heads > 1 and s1 != d):
        raise ValueError(f"{name} needs contiguous rows (any row stride) on the cache's device")
    return s0 if m > 1 else heads * d


def _i32(t, name: str, count: int, cache: svp_cache) -> int:
    """Address of a contiguous int32 vector of at least ``count`` entries (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.get_device() != cache.index or not t.is_contiguous() or t.numel() < count:
        raise ValueError(f"{name} must be {count} or more contiguous int32 values on the cache's device")
    return t.data_ptr()


def _requests(cu, cache: svp_cache, name: str) -> int:
    """Number of requests of cu [n+1]."""
    n = cu.numel() - 1
    if n < 0 or n > cache.max_n:
        raise ValueError(f"{name} must have 1..{cache.max_n + 1} entries (rows of the block table)")
    if cache.index != torch._C._cuda_getDevice():
        raise ValueError("the cache must be on the current CUDA device")
    return n


def _raw_stream(stream, cache: svp_cache) -> int:
    return torch._C._cuda_getCurrentRawStream(cache.index) if stream is None else _stream(stream)


def _other_stream(stream, cache: svp_cache):
    """Context that makes ``stream`` torch's current one, None if it is: what a call allocates, clears
    or captures belongs to the stream that it runs on."""
    raw = _raw_stream(stream, cache)
    if stream is None or raw == torch._C._cuda_getCurrentRawStream(cache.index):
        return None
    return torch.cuda.stream(torch.cuda.ExternalStream(raw, cache.device) if raw else
                             torch.cuda.default_stream(cache.device))


def _cache_workspace(cache: svp_cache, stream) -> Workspace:
    """Status word of cache_write / cache_read calls that bring no workspace: nothing else is
    kept there, so every stream and graph may share it."""
    ws = cache.ws
    if ws is None:
        ws = cache.ws = _workspace(("cache",), 256, cache.device, stream)
    return ws


def cache_write(k, v, ctx_len, cu_slots, *, cache: svp_cache, take=None,
                ws: Optional[Workspace] = None, stream=None) -> None:
    """Store packed rows k, v [m_cap, hkv, d] (bf16 or fp32; slices of a fused projection are
    fine) at positions ctx_len[i] + j of their requests (svp_cache_write).  take [n] int32:
    only the first take[i] rows of request i, e.g. the accept_len of margin_accept.  ws: 256
    bytes for the device status, which a call without one does not report."""
    n = _requests(cu_slots, cache, "cu_slots")
    stride = _rows(k, "k", cache.hkv, cache)
    if k.dtype is not v.dtype or _rows(v, "v", cache.hkv, cache) != stride or k.numel() != v.numel():
        raise ValueError("k and v need one shape, type and row stride")
    if ws is None:
        ws = _cache_workspace(cache, stream)
    st = lib().svp_cache_write(
        k.data_ptr(), v.data_ptr(), stride, _dtype_code(k), cache, _i32(ctx_len, "ctx_len", n, cache),
        _i32(cu_slots, "cu_slots", n + 1, cache), _i32(take, "take", n, cache), n, k.shape[0], cache.hkv,
        cache.d, ws.ptr, ws.nbytes, _raw_stream(stream, cache))
    if st:
        raise SvpError(st, "svp_cache_write")


def cache_read(start, cu_rows, *, cache: svp_cache, rows: Optional[int] = None,
               dtype: torch.dtype = torch.bfloat16, k_out=None, v_out=None,
               ws: Optional[Workspace] = None, stream=None):
    """Positions start[i].. (0.. for None) of each request as contiguous rows
    cu_rows[i]..cu_rows[i+1]-1 of (k_out, v_out) [rows, hkv, d] (svp_cache_read).  Outputs that
    are not given are made with ``rows`` rows of ``dtype``, zeros where nothing is read.  ws as for
    cache_write."""
    n = _requests(cu_rows, cache, "cu_rows")
    dev = cache.device
    other = _other_stream(stream, cache)
    if other is not None:
        with other:
            return cache_read(start, cu_rows, cache=cache, rows=rows, dtype=dtype, k_out=k_out, v_out=v_out, ws=ws)
    if k_out is None or v_out is None:
        if rows is None or k_out is not None or v_out is not None:
            raise ValueError("give both k_out and v_out, or rows")
        k_out = torch.zeros(rows, cache.hkv, cache.d, dtype=dtype, device=dev)
        v_out = torch.zeros_like(k_out)
    _rows(k_out, "k_out", cache.hkv, cache)
    _rows(v_out, "v_out", cache.hkv, cache)
    if (k_out.shape != v_out.shape or k_out.dtype != v_out.dtype or not k_out.is_contiguous()
            or not v_out.is_contiguous()):
        raise ValueError("k_out and v_out must be contiguous, of one shape and type")
    if ws is None:
        ws = _cache_workspace(cache, stream)
    st = lib().svp_cache_read(
        cache, _i32(start, "start", n, cache), _i32(cu_rows, "cu_rows", n + 1, cache), n, k_out.shape[0],
        cache.hkv, cache.d, _dtype_code(k_out), k_out.data_ptr(), v_out.data_ptr(), ws.ptr, ws.nbytes,
        _raw_stream(stream, cache))
    if st:
        raise SvpError(st, "svp_cache_read")
    return k_out, v_out


def chunk_attn_workspace_size(hq: int, hkv: int, d: int, dtype=torch.bfloat16) -> int:
    nb = ctypes.c_size_t(0)
    h = _heads(hq, hkv, d, 0.0)
    _check(lib().svp_chunk_attn_workspace_size(ctypes.byref(h), SVP_BF16 if dtype == torch.bfloat16 else SVP_F32,
                                               ctypes.byref(nb)), "svp_chunk_attn_workspace_size")
    return int(nb.value)


_chunk_ws: dict = {}
_CHUNK_WS_MOST = 16       # scratch buffers kept (20 MB each at d = 64, else 40)


def _chunk_workspace(hq: int, cache: svp_cache, dtype, raw: int) -> Workspace:
    """The scratch of chunk_attn calls that bring none: one for each stream, as calls on two
    streams may overlap; a call that is being captured gets its own, which lives in the memory
    pool that torch.cuda.graph gives the graph, as graphs may be replayed on any stream (and is not zeroed, as its status word, which
    kernels only add bits to, is out of reach)."""
    if torch._C._cuda_isCurrentStreamCapturing():
        return Workspace(chunk_attn_workspace_size(hq, cache.hkv, cache.d, dtype), cache.device, zeroed=0)
    key = (raw, cache.index, cache.d, dtype)
    ws = _chunk_ws.get(key)
    if ws is None:
        while len(_chunk_ws) >= _CHUNK_WS_MOST:
            # (the oldest; torch's allocator gives its memory to later work of its own stream only)
            _chunk_ws.pop(next(iter(_chunk_ws)), None)
        ws = _chunk_ws[key] = Workspace(chunk_attn_workspace_size(hq, cache.hkv, cache.d, dtype),
                                        cache.device, zeroed=256)
    return ws


def chunk_attn(q, ctx_len, cu_slots, *, cache: svp_cache, w: Optional[int] = None, out=None,
               lse=None, want_lse: bool = True, scale: float = 0.0, ws: Optional[Workspace] = None,
               stream=None):
    """Attention of packed new rows q [m_cap, hq, d] over the cache; row j of request i sees
    positions 0..ctx_len[i]+j, its own (written by cache_write before) included.  w: largest
    row count of a request (default m_cap; calls of few rows are planned by it).  Returns
    (out [m_cap, hq, d], lse [m_cap, hq] or None); rows past cu_slots[n] are left as they were
    (zeros in outputs made here).

    ws: a Workspace of chunk_attn_workspace_size bytes.  Without one the call takes scratch kept for
    its stream, whose device status nobody can read: what has to see skipped requests, bad pages or
    time-outs brings ws and asks ws.read_status.  So does a capture begun otherwise than by
    torch.cuda.graph (or CUDAGraph.capture_begin), as only there the scratch belongs to the graph, and
    work on a stream that is destroyed before it has run, as a later stream may get the same handle."""
    n = _requests(cu_slots, cache, "cu_slots")
    other = _other_stream(stream, cache)
    if other is not None:
        with other:
            return chunk_attn(q, ctx_len, cu_slots, cache=cache, w=w, out=out, lse=lse, want_lse=want_lse,
                              scale=scale, ws=ws)
    dev = cache.device
    hkv = cache.hkv
    m_cap, hq, d = q.shape
    if hq < 1 or hq % hkv:
        raise ValueError("the query heads must be a multiple of the cache's heads")
    stride = _rows(q, "q", hq, cache)
    if out is None:
        out = torch.zeros(m_cap, hq, d, dtype=q.dtype, device=dev)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be contiguous, of q's shape, type and device")
    if lse is None:
        if want_lse:
            lse = torch.zeros(m_cap, hq, dtype=torch.float32, device=dev)
    elif lse.shape != (m_cap, hq) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [m_cap, hq] on q's device")
    raw = _raw_stream(None, cache)
    if ws is None:
        ws = _chunk_workspace(hq, cache, q.dtype, raw)
    st = lib().svp_chunk_attn(
        q.data_ptr(), stride, cache, _i32(ctx_len, "ctx_len", n, cache), _i32(cu_slots, "cu_slots", n + 1, cache),
        n, m_cap, (m_cap or 1) if w is None else w, svp_heads(hq, hkv, d, scale), _dtype_code(q), out.data_ptr(),
        0 if lse is None else lse.data_ptr(), ws.ptr, ws.nbytes, raw)
    if st:
        raise SvpError(st, "svp_chunk_attn")
    return out, lse
