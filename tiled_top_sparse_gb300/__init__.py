"""Thin Python binding over libtts.so (the C ABI declared in include/tts.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. There is
no fallback: if the library (or, for the grouped-query calls, the CPython module
built beside it) is missing or fails to load, calls raise.

    attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                    causal, scale, out=None, lse=None, workspace=None, status=None)
    attn_fwd_varlen_window(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                           window, sinks, scale, out=None, lse=None, workspace=None, status=None)
    topk_select(logits, row_starts, row_lens, k, idx=None, status=None)
    sparse_attn_paged(q, kv_cache, page_table, idx, kv_len, scale, dv=512,
                      out=None, lse=None, status=None)
    quantize_fp8_prefill(q, k)
    attn_fwd_varlen_fp8(q8, q_scale, k8, k_scale, v, cu_seqlens_q, cu_seqlens_k,
                        max_seqlen_q, max_seqlen_k, causal, scale, out=None, lse=None,
                        workspace=None, status=None)
    rope_kv_append(k, v, k_cache, v_cache, page_tables, past_lens, cu_new, max_new,
                   k_scale=None, v_scale=None, cos_sin=None, q=None, q_out=None, k_out=None,
                   status=None)
    attn_decode_paged(q, k_cache, v_cache, page_tables, kv_lens, scale, cu_seqlens_q=None,
                      max_seqlen_q=1, k_scale=None, v_scale=None, window=0, sinks=0, out=None,
                      lse=None, workspace=None, status=None)
    rope_kv_append_axes(k, v, k_cache, v_cache, page_tables, past_lens, cu_new, max_new,
                        positions, pair_axis, cos_sin, k_scale=None, v_scale=None, q=None,
                        q_out=None, k_out=None, status=None)
    attn_decode_tree(q, k_cache, v_cache, page_tables, kv_lens, tree_mask, scale, cu_seqlens_q,
                     max_seqlen_q, k_scale=None, v_scale=None, window=0, sinks=0, out=None,
                     lse=None, workspace=None, status=None)
    kv_compact(k_cache, v_cache, page_tables, past_lens, path, path_lens, k_scale=None,
               v_scale=None, kv_lens=None, status=None)
    kv_fork(k_cache, v_cache, page_tables, kv_lens, parents, new_pages, k_scale=None,
            v_scale=None, tables_out=None, lens_out=None, status=None)
    rope_axes(sections, interleaved=False)
    rope_cache(max_pos, rot_dim, base=10000.0, out=None, device=None)
    qkv_rope(x, w, bias, positions, cos_sin, num_heads, q=None, k=None, v=None,
             status=None)
    qkv_rope_axes(x, w, bias, positions, pair_axis, cos_sin, num_heads, q=None, k=None, v=None,
                  status=None)

`status`, when given, is a 1-element int32 CUDA tensor the kernels OR their
device-side flags into (see TTS_DEV_* in the header); `check_status(status)`
synchronises and raises on a set flag.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtts.so")

TTS_OK = 0
TTS_ERR_INVALID_ARG = 1
TTS_ERR_UNSUPPORTED = 2
TTS_ERR_CUDA = 3
TTS_ERR_INDEX_RANGE = 4
TTS_ERR_DEVICE_TIMEOUT = 5
TTS_ERR_WORKSPACE = 6
TTS_BF16 = 0
TTS_F32 = 1
TTS_E4M3 = 2
TTS_DEV_INDEX_RANGE = 0x1
TTS_DEV_TIMEOUT = 0x2
TTS_DEV_BAD_ARG = 0x4

EXPORTED = (
    "tts_status_string",
    "tts_status_from_device",
    "tts_version",
    "tts_attn_workspace_bytes",
    "tts_attn_fwd_varlen",
    "tts_attn_fwd_varlen_window",
    "tts_topk_select",
    "tts_topk_long_workspace_bytes",
    "tts_topk_select_long",
    "tts_sparse_attn_paged",
    "tts_sparse_workspace_bytes",
    "tts_sparse_attn_decode",
    "tts_paged_kv_write",
    "tts_quantize_fp8_prefill",
    "tts_attn_fwd_varlen_fp8",
    "tts_rope_kv_append",
    "tts_rope_kv_append_axes",
    "tts_kv_compact",
    "tts_kv_fork",
    "tts_attn_decode_workspace_bytes",
    "tts_attn_decode_paged",
    "tts_attn_decode_tree_workspace_bytes",
    "tts_attn_decode_tree",
    "tts_rope_cache",
    "tts_qkv_rope",
    "tts_qkv_rope_axes",
    "tts_attn_fwd_varlen_f32_noalloc",
    "tts_debug_wait_timeout",
)


class TTSError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} (code {code})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libtts.so (built by tiled_top_sparse_gb300._build). Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libtts.so not built ({LIB_PATH}); run tiled_top_sparse_gb300/_build.py")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    L.tts_status_string.argtypes = [ctypes.c_int]
    L.tts_status_string.restype = ctypes.c_char_p
    L.tts_status_from_device.argtypes = [ctypes.c_uint32]
    L.tts_status_from_device.restype = ctypes.c_int
    L.tts_version.argtypes = []
    L.tts_version.restype = ctypes.c_int
    L.tts_attn_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, ctypes.c_int]
    L.tts_attn_workspace_bytes.restype = ctypes.c_size_t
    L.tts_attn_fwd_varlen.argtypes = [P, P, P, ctypes.c_int, i64, i64, P, P, i32, i32, i32, i32,
                                      i32, i32, i32, f32, P, P, P, ctypes.c_size_t, P, P]
    L.tts_attn_fwd_varlen.restype = ctypes.c_int
    L.tts_attn_fwd_varlen_window.argtypes = [P, P, P, ctypes.c_int, i64, i64, P, P, i32, i32, i32,
                                             i32, i32, i32, i32, i32, f32, P, ctypes.c_int, P, P,
                                             ctypes.c_size_t, P, P]
    L.tts_attn_fwd_varlen_window.restype = ctypes.c_int
    L.tts_topk_select.argtypes = [P, i64, i32, P, P, i32, P, P, P]
    L.tts_topk_select.restype = ctypes.c_int
    L.tts_topk_long_workspace_bytes.argtypes = [i32, i64, i32]
    L.tts_topk_long_workspace_bytes.restype = ctypes.c_size_t
    L.tts_topk_select_long.argtypes = [P, i64, i32, P, P, i32, P, P, ctypes.c_size_t, P, P]
    L.tts_topk_select_long.restype = ctypes.c_int
    L.tts_sparse_attn_paged.argtypes = [P, i32, i32, i32, i32, P, i32, i32, P, i32, i32, P, i32,
                                        f32, P, P, P, ctypes.c_size_t, P, P]
    L.tts_sparse_attn_paged.restype = ctypes.c_int
    L.tts_sparse_attn_decode.argtypes = [P, i32, i32, i32, i32, P, i32, i32, P, i32, P, P, i32,
                                         f32, P, P, P, ctypes.c_size_t, P, P]
    L.tts_sparse_attn_decode.restype = ctypes.c_int
    L.tts_paged_kv_write.argtypes = [P, i64, i32, P, P, P, i32, i32, P, i32, i32, P, P]
    L.tts_paged_kv_write.restype = ctypes.c_int
    L.tts_sparse_workspace_bytes.argtypes = [i32]
    L.tts_sparse_workspace_bytes.restype = ctypes.c_size_t
    L.tts_quantize_fp8_prefill.argtypes = [P, i64, i32, P, i64, i32, i32, P, P, P, P, P]
    L.tts_quantize_fp8_prefill.restype = ctypes.c_int
    L.tts_attn_fwd_varlen_fp8.argtypes = [P, P, P, P, P, i64, i64, P, P, i32, i32, i32, i32,
                                          i32, i32, i32, f32, P, P, P, ctypes.c_size_t, P, P]
    L.tts_attn_fwd_varlen_fp8.restype = ctypes.c_int
    L.tts_rope_kv_append.argtypes = [P, i64, i32, P, i64, P, i64, i64, P, P, i32, i32, i32, i32, P,
                                     i32, P, i32, P, P, P, P, ctypes.c_int, i32, i32, P, P, P, P]
    L.tts_rope_kv_append.restype = ctypes.c_int
    L.tts_attn_decode_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.tts_attn_decode_workspace_bytes.restype = ctypes.c_size_t
    L.tts_attn_decode_paged.argtypes = [P, i64, P, i32, i32, i32, i32, i32, P, P, P, P,
                                        ctypes.c_int, i32, i32, P, i32, P, i32, i32, f32, P,
                                        ctypes.c_int, P, P, ctypes.c_size_t, P, P]
    L.tts_attn_decode_paged.restype = ctypes.c_int
    L.tts_rope_kv_append_axes.argtypes = [
        P, i64, i32, P, i64, P, i64, i64, P, P, i32, i32, i32, i32, P, i32, P, i32, ctypes.c_char_p,
        P, i32, P, P, P, P, ctypes.c_int, i32, i32, P, P, P, P]
    L.tts_rope_kv_append_axes.restype = ctypes.c_int
    L.tts_kv_compact.argtypes = [P, P, P, P, ctypes.c_int, i32, i32, i32, i32, P, i32, P, i32, P,
                                 i32, P, P, P, P]
    L.tts_kv_compact.restype = ctypes.c_int
    L.tts_kv_fork.argtypes = [P, P, P, P, ctypes.c_int, i32, i32, i32, i32, P, i32, P, i32, P, P,
                              i32, P, P, P, P]
    L.tts_kv_fork.restype = ctypes.c_int
    L.tts_attn_decode_tree_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.tts_attn_decode_tree_workspace_bytes.restype = ctypes.c_size_t
    L.tts_attn_decode_tree.argtypes = [P, i64, P, P, i32, i32, i32, i32, i32, P, P, P, P,
                                       ctypes.c_int, i32, i32, P, i32, P, i32, i32, f32, P,
                                       ctypes.c_int, P, P, ctypes.c_size_t, P, P]
    L.tts_attn_decode_tree.restype = ctypes.c_int
    L.tts_qkv_rope_axes.argtypes = [P, i64, i32, P, P, P, i32, ctypes.c_char_p, P, i32, i32, i32,
                                    P, P, P, P, P]
    L.tts_qkv_rope_axes.restype = ctypes.c_int
    L.tts_rope_cache.argtypes = [i32, i32, f32, P, P]
    L.tts_rope_cache.restype = ctypes.c_int
    L.tts_qkv_rope.argtypes = [P, i64, i32, P, P, P, P, i32, i32, i32, P, P, P, P, P]
    L.tts_qkv_rope.restype = ctypes.c_int
    L.tts_attn_fwd_varlen_f32_noalloc.argtypes = [P, P, P, i64, i64, P, P, i32, i32, i32, i32,
                                                  i32, i32, i32, f32, P, P, P, P]
    L.tts_attn_fwd_varlen_f32_noalloc.restype = ctypes.c_int
    L.tts_debug_wait_timeout.argtypes = [P, P]
    L.tts_debug_wait_timeout.restype = ctypes.c_int
    _lib = L
    return L


def status_string(code: int) -> str:
    return lib().tts_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(code: int, what: str):
    if code != TTS_OK:
        raise TTSError(code, what)


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _cuda_contig(t: torch.Tensor, name: str, dtype=None):
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    if dtype is not None:
        _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")


def check_status(status: torch.Tensor, what: str = "device status"):
    """Synchronise on `status` (1-element int32 CUDA tensor) and raise if a flag is set."""
    v = int(status.item()) & 0xFFFFFFFF
    _check(lib().tts_status_from_device(ctypes.c_uint32(v)), what)


def debug_wait_timeout(status: torch.Tensor):
    """Run the library's bounded-wait self-test kernel (see tts_debug_wait_timeout)."""
    _cuda_contig(status, "status", torch.int32)
    _check(lib().tts_debug_wait_timeout(_ptr(status), _stream(status.device)),
           "tts_debug_wait_timeout")


def attn_workspace_bytes(total_q, total_k, num_heads_q, num_heads_kv, head_dim, dtype) -> int:
    code = TTS_F32 if dtype == torch.float32 else TTS_BF16
    return int(lib().tts_attn_workspace_bytes(int(total_q), int(total_k), int(num_heads_q),
                                              int(num_heads_kv), int(head_dim), code))


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal,
                    scale, out=None, lse=None, workspace=None, status=None, want_lse=True):
    """Dense attention forward over packed varlen sequences (tts_attn_fwd_varlen).

    q [total_q, Hq, d], k/v [total_k, Hkv, d] (bf16 or fp32, same dtype), cu_seqlens_* int32
    [batch+1] on the device. Returns (out fp32 [total_q, Hq, d], lse fp32 [total_q, Hq]).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _cuda_contig(t, n)
        _need(t.dim() == 3, f"{n} must be [tokens, heads, head_dim]")
    _need(q.dtype == k.dtype == v.dtype and q.dtype in (torch.bfloat16, torch.float32),
          "q, k, v must share dtype bf16 or fp32")
    _need(k.shape == v.shape, "k and v must have the same shape")
    _cuda_contig(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    _cuda_contig(cu_seqlens_k, "cu_seqlens_k", torch.int32)
    total_q, hq, d = q.shape
    total_k, hkv, d2 = k.shape
    _need(d == d2, "head_dim mismatch")
    batch = cu_seqlens_q.numel() - 1
    _need(batch >= 1 and cu_seqlens_k.numel() == batch + 1, "cu_seqlens sizes must be batch+1")
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=torch.float32, device=q.device)
    _cuda_contig(out, "out", torch.float32)
    _need(tuple(out.shape) == (total_q, hq, d), "out shape")
    if lse is None and want_lse:
        lse = torch.empty((total_q, hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _cuda_contig(lse, "lse", torch.float32)
    dt = TTS_F32 if q.dtype == torch.float32 else TTS_BF16
    need = attn_workspace_bytes(total_q, total_k, hq, hkv, d, q.dtype)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    code = lib().tts_attn_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), dt, total_q, total_k, _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
        batch, int(max_seqlen_q), int(max_seqlen_k), hq, hkv, d, int(bool(causal)), float(scale),
        _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status), _stream(q.device))
    _check(code, "tts_attn_fwd_varlen")
    return out, lse


def attn_fwd_varlen_window(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, window,
                           sinks, scale, out=None, lse=None, workspace=None, status=None,
                           want_lse=True, out_dtype=torch.float32):
    """Causal sliding-window attention with first tokens that stay visible
    (tts_attn_fwd_varlen_window): a row sees the last `window` keys up to its own position and
    the first `sinks`.

    Arguments as attn_fwd_varlen; returns (out [total_q, Hq, d] in out_dtype, or in out's dtype:
    fp32 or bf16; lse fp32 [total_q, Hq])."""
    out, lse = _attn_outputs(q, out, lse, want_lse, out_dtype)
    call = (_nat or _binding()).attn_fwd_varlen_window
    code = call(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, window, sinks,
                scale, out, lse, workspace, status)
    if code == TTS_ERR_WORKSPACE:  # missing or too small: nothing was enqueued
        need = attn_workspace_bytes(q.shape[0], k.shape[0], q.shape[1], k.shape[1], q.shape[2],
                                    q.dtype)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        code = call(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, window,
                    sinks, scale, out, lse, workspace, status)
    if code:
        raise TTSError(code, "tts_attn_fwd_varlen_window")
    return out, lse


def topk_select(logits, row_starts, row_lens, k, idx=None, status=None):
    """Deterministic per-row top-k (tts_topk_select). Returns idx int32 [rows, k]."""
    _cuda_contig(logits, "logits", torch.float32)
    _need(logits.dim() == 2, "logits must be [rows, row_stride]")
    _cuda_contig(row_starts, "row_starts", torch.int32)
    _cuda_contig(row_lens, "row_lens", torch.int32)
    rows, stride = logits.shape
    _need(row_starts.numel() == rows and row_lens.numel() == rows, "row_starts/row_lens size")
    if idx is None:
        idx = torch.empty((rows, int(k)), dtype=torch.int32, device=logits.device)
    _cuda_contig(idx, "idx", torch.int32)
    _need(tuple(idx.shape) == (rows, int(k)), "idx shape")
    code = lib().tts_topk_select(_ptr(logits), stride, rows, _ptr(row_starts), _ptr(row_lens),
                                 int(k), _ptr(idx), _ptr(status), _stream(logits.device))
    _check(code, "tts_topk_select")
    return idx


def topk_long_workspace_bytes(rows, row_stride, k) -> int:
    return int(lib().tts_topk_long_workspace_bytes(int(rows), int(row_stride), int(k)))


def topk_select_long(logits, row_starts, row_lens, k, idx=None, workspace=None, status=None):
    """Deterministic top-k over long rows (tts_topk_select_long): the same result as
    topk_select for rows up to 2^30 values. Returns idx int32 [rows, k]. A workspace of
    topk_long_workspace_bytes(...) bytes is allocated here when `workspace` is missing."""
    _cuda_contig(logits, "logits", torch.float32)
    _need(logits.dim() == 2, "logits must be [rows, row_stride]")
    _cuda_contig(row_starts, "row_starts", torch.int32)
    _cuda_contig(row_lens, "row_lens", torch.int32)
    rows, stride = logits.shape
    _need(row_starts.numel() == rows and row_lens.numel() == rows, "row_starts/row_lens size")
    if idx is None:
        idx = torch.empty((rows, int(k)), dtype=torch.int32, device=logits.device)
    _cuda_contig(idx, "idx", torch.int32)
    _need(tuple(idx.shape) == (rows, int(k)), "idx shape")
    need = topk_long_workspace_bytes(rows, stride, k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=logits.device)
    _cuda_contig(workspace, "workspace", torch.uint8)
    code = lib().tts_topk_select_long(_ptr(logits), stride, rows, _ptr(row_starts),
                                      _ptr(row_lens), int(k), _ptr(idx), _ptr(workspace),
                                      workspace.numel(), _ptr(status), _stream(logits.device))
    _check(code, "tts_topk_select_long")
    return idx


def sparse_attn_decode(q, kv_cache, page_tables, kv_lens, idx, scale, dv=512, out=None,
                       lse=None, workspace=None, status=None, want_lse=True, split=True):
    """Decode-shaped sparse attention (tts_sparse_attn_decode): one query per request,
    request n reading through page_tables[n] with length kv_lens[n].

    q bf16 [nreq, H, dqk], kv_cache bf16 [pages, page_size, dqk], page_tables int32
    [nreq, max_pages], kv_lens int32 [nreq], idx int32 [nreq, topk]. Returns (out fp32
    [nreq, H, dv], lse fp32 [nreq, H]); `split` as in sparse_attn_paged."""
    _cuda_contig(q, "q", torch.bfloat16)
    _cuda_contig(kv_cache, "kv_cache", torch.bfloat16)
    _cuda_contig(page_tables, "page_tables", torch.int32)
    _cuda_contig(kv_lens, "kv_lens", torch.int32)
    _cuda_contig(idx, "idx", torch.int32)
    _need(q.dim() == 3 and kv_cache.dim() == 3 and idx.dim() == 2 and page_tables.dim() == 2,
          "ranks")
    nreq, H, dqk = q.shape
    pages, page_size, dk2 = kv_cache.shape
    _need(dk2 == dqk and idx.shape[0] == nreq and page_tables.shape[0] == nreq and
          kv_lens.numel() == nreq, "shapes")
    if out is None:
        out = torch.empty((nreq, H, dv), dtype=torch.float32, device=q.device)
    _cuda_contig(out, "out", torch.float32)
    if lse is None and want_lse:
        lse = torch.empty((nreq, H), dtype=torch.float32, device=q.device)
    ws_bytes = 0
    if split:
        need = sparse_workspace_bytes(nreq)
        if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    else:
        workspace = None
    code = lib().tts_sparse_attn_decode(
        _ptr(q), nreq, H, dqk, int(dv), _ptr(kv_cache), pages, page_size, _ptr(page_tables),
        page_tables.shape[1], _ptr(kv_lens), _ptr(idx), idx.shape[1], float(scale), _ptr(out),
        _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status), _stream(q.device))
    _check(code, "tts_sparse_attn_decode")
    return out, lse


def paged_kv_write(kv_cache, page_tables, kv_new, positions, req_ids=None, status=None):
    """Write rows into the paged KV cache (tts_paged_kv_write): token t's row kv_new[t]
    goes to its request's page at logical position positions[t]. In place; returns
    kv_cache."""
    _cuda_contig(kv_cache, "kv_cache", torch.bfloat16)
    _cuda_contig(page_tables, "page_tables", torch.int32)
    _cuda_contig(kv_new, "kv_new", torch.bfloat16)
    _cuda_contig(positions, "positions", torch.int32)
    if req_ids is not None:
        _cuda_contig(req_ids, "req_ids", torch.int32)
    _need(kv_cache.dim() == 3 and kv_new.dim() == 2 and page_tables.dim() == 2, "ranks")
    pages, page_size, dim = kv_cache.shape
    ntok = kv_new.shape[0]
    _need(kv_new.shape[1] == dim and positions.numel() == ntok and
          (req_ids is None or req_ids.numel() == ntok), "shapes")
    code = lib().tts_paged_kv_write(_ptr(kv_new), ntok, dim, _ptr(req_ids), _ptr(positions),
                                    _ptr(page_tables), page_tables.shape[1],
                                    page_tables.shape[0], _ptr(kv_cache), pages, page_size,
                                    _ptr(status), _stream(kv_new.device))
    _check(code, "tts_paged_kv_write")
    return kv_cache


def sparse_workspace_bytes(nq) -> int:
    return int(lib().tts_sparse_workspace_bytes(int(nq)))


def sparse_attn_paged(q, kv_cache, page_table, idx, kv_len, scale, dv=512, out=None, lse=None,
                      workspace=None, status=None, want_lse=True, split=True):
    """Order-invariant sparse attention through a page table (tts_sparse_attn_paged).

    q bf16 [nq, H, dqk], kv_cache bf16 [pages, page_size, dqk], page_table int32 [n_pages],
    idx int32 [nq, topk]. Returns (out fp32 [nq, H, dv], lse fp32 [nq, H]). With split
    (default) a workspace for the split of the last wave is passed (allocated here when
    `workspace` is missing or too small); split=False passes none.
    """
    _cuda_contig(q, "q", torch.bfloat16)
    _cuda_contig(kv_cache, "kv_cache", torch.bfloat16)
    _cuda_contig(page_table, "page_table", torch.int32)
    _cuda_contig(idx, "idx", torch.int32)
    _need(q.dim() == 3 and kv_cache.dim() == 3 and idx.dim() == 2, "ranks")
    nq, H, dqk = q.shape
    pages, page_size, dk2 = kv_cache.shape
    _need(dk2 == dqk and idx.shape[0] == nq, "shapes")
    if out is None:
        out = torch.empty((nq, H, dv), dtype=torch.float32, device=q.device)
    _cuda_contig(out, "out", torch.float32)
    if lse is None and want_lse:
        lse = torch.empty((nq, H), dtype=torch.float32, device=q.device)
    ws_bytes = 0
    if split:
        need = sparse_workspace_bytes(nq)
        if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    else:
        workspace = None
    code = lib().tts_sparse_attn_paged(
        _ptr(q), nq, H, dqk, int(dv), _ptr(kv_cache), pages, page_size, _ptr(page_table),
        page_table.numel(), int(kv_len), _ptr(idx), idx.shape[1], float(scale), _ptr(out),
        _ptr(lse), _ptr(workspace), ws_bytes, _ptr(status), _stream(q.device))
    _check(code, "tts_sparse_attn_paged")
    return out, lse


def rope_cache(max_pos, rot_dim, base=10000.0, out=None, device=None):
    """cos/sin table of rotary embedding (tts_rope_cache): fp32 [max_pos, rot_dim/2, 2]
    holding (cos, sin) of p * base^(-2j/rot_dim)."""
    if out is None:
        dev = torch.device("cuda") if device is None else torch.device(device)
        out = torch.empty((int(max_pos), int(rot_dim) // 2, 2), dtype=torch.float32, device=dev)
    _cuda_contig(out, "out", torch.float32)
    _need(tuple(out.shape) == (int(max_pos), int(rot_dim) // 2, 2), "out shape")
    code = lib().tts_rope_cache(int(max_pos), int(rot_dim), float(base), _ptr(out),
                                _stream(out.device))
    _check(code, "tts_rope_cache")
    return out


def qkv_rope(x, w, bias, positions, cos_sin, num_heads, q=None, k=None, v=None, status=None):
    """Vision QKV projection + RoPE (tts_qkv_rope).

    x bf16 [n, hidden], w bf16 [3*H*d, hidden], bias fp32 [3*H*d] or None, positions
    int32 [n], cos_sin fp32 [max_pos, d/2, 2] (rope_cache with rot_dim = d). Returns
    (q, k, v) bf16 [n, H, d]: q and k rotated, v as projected."""
    _cuda_contig(x, "x", torch.bfloat16)
    _cuda_contig(w, "w", torch.bfloat16)
    _cuda_contig(positions, "positions", torch.int32)
    _cuda_contig(cos_sin, "cos_sin", torch.float32)
    _need(x.dim() == 2 and w.dim() == 2 and w.shape[1] == x.shape[1], "x [n, hidden], "
          "w [3*H*d, hidden]")
    n, hidden = x.shape
    H = int(num_heads)
    _need(w.shape[0] % (3 * H) == 0, "w rows must be 3 * num_heads * head_dim")
    d = w.shape[0] // (3 * H)
    _need(positions.numel() == n, "positions size")
    _need(cos_sin.dim() == 3 and cos_sin.shape[1] == d // 2 and cos_sin.shape[2] == 2,
          "cos_sin must be [max_pos, head_dim/2, 2]")
    if bias is not None:
        _cuda_contig(bias, "bias", torch.float32)
        _need(bias.numel() == 3 * H * d, "bias size")
    outs = []
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t is None:
            t = torch.empty((n, H, d), dtype=torch.bfloat16, device=x.device)
        _cuda_contig(t, name, torch.bfloat16)
        _need(tuple(t.shape) == (n, H, d), f"{name} shape")
        outs.append(t)
    code = lib().tts_qkv_rope(_ptr(x), n, hidden, _ptr(w), _ptr(bias), _ptr(positions),
                              _ptr(cos_sin), cos_sin.shape[0], H, d, _ptr(outs[0]),
                              _ptr(outs[1]), _ptr(outs[2]), _ptr(status), _stream(x.device))
    _check(code, "tts_qkv_rope")
    return tuple(outs)


def quantize_fp8_prefill(q, k, q8=None, q_scale=None, k8=None, k_scale=None):
    """e4m3 block quantization (tts_quantize_fp8_prefill) of q bf16 [Tq, Hq, d] (scale per
    token and head) and k bf16 [Tk, Hkv, d] (scale per KV head). Returns (q8, q_scale, k8,
    k_scale): codes as uint8 tensors of the input shapes (view them as
    torch.float8_e4m3fn to read values), scales fp32 [Tq, Hq] and [Hkv]."""
    _cuda_contig(q, "q", torch.bfloat16)
    _cuda_contig(k, "k", torch.bfloat16)
    _need(q.dim() == 3 and k.dim() == 3 and q.shape[2] == k.shape[2], "q, k [tokens, heads, d]")
    tq, hq, d = q.shape
    tk, hkv, _ = k.shape
    dev = q.device
    q8 = torch.empty((tq, hq, d), dtype=torch.uint8, device=dev) if q8 is None else q8
    k8 = torch.empty((tk, hkv, d), dtype=torch.uint8, device=dev) if k8 is None else k8
    q_scale = torch.empty((tq, hq), dtype=torch.float32, device=dev) if q_scale is None else q_scale
    k_scale = torch.empty((hkv,), dtype=torch.float32, device=dev) if k_scale is None else k_scale
    for t, n, dt in ((q8, "q8", torch.uint8), (k8, "k8", torch.uint8),
                     (q_scale, "q_scale", torch.float32), (k_scale, "k_scale", torch.float32)):
        _cuda_contig(t, n, dt)
    code = lib().tts_quantize_fp8_prefill(_ptr(q), tq, hq, _ptr(k), tk, hkv, d, _ptr(q8),
                                          _ptr(q_scale), _ptr(k8), _ptr(k_scale),
                                          _stream(dev))
    _check(code, "tts_quantize_fp8_prefill")
    return q8, q_scale, k8, k_scale


def attn_fwd_varlen_fp8(q8, q_scale, k8, k_scale, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                        max_seqlen_k, causal, scale, out=None, lse=None, workspace=None,
                        status=None, want_lse=True):
    """Dense attention with e4m3 q / k in Q K^T (tts_attn_fwd_varlen_fp8). q8 / k8 uint8
    codes [T, H, 128] with their scales from quantize_fp8_prefill, v bf16. Returns (out
    fp32 [Tq, Hq, 128], lse fp32 [Tq, Hq])."""
    _cuda_contig(q8, "q8", torch.uint8)
    _cuda_contig(k8, "k8", torch.uint8)
    _cuda_contig(q_scale, "q_scale", torch.float32)
    _cuda_contig(k_scale, "k_scale", torch.float32)
    _cuda_contig(v, "v", torch.bfloat16)
    _cuda_contig(cu_seqlens_q, "cu_seqlens_q", torch.int32)
    _cuda_contig(cu_seqlens_k, "cu_seqlens_k", torch.int32)
    _need(q8.dim() == 3 and k8.shape == v.shape, "q8 [Tq, Hq, d]; k8, v [Tk, Hkv, d]")
    total_q, hq, d = q8.shape
    total_k, hkv, _ = k8.shape
    _need(tuple(q_scale.shape) == (total_q, hq) and k_scale.numel() == hkv, "scale shapes")
    batch = cu_seqlens_q.numel() - 1
    _need(batch >= 1 and cu_seqlens_k.numel() == batch + 1, "cu_seqlens sizes must be batch+1")
    if out is None:
        out = torch.empty((total_q, hq, d), dtype=torch.float32, device=q8.device)
    _cuda_contig(out, "out", torch.float32)
    if lse is None and want_lse:
        lse = torch.empty((total_q, hq), dtype=torch.float32, device=q8.device)
    need = attn_workspace_bytes(total_q, total_k, hq, hkv, d, torch.bfloat16)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q8.device)
    code = lib().tts_attn_fwd_varlen_fp8(
        _ptr(q8), _ptr(q_scale), _ptr(k8), _ptr(k_scale), _ptr(v), total_q, total_k,
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch, int(max_seqlen_q), int(max_seqlen_k), hq,
        hkv, d, int(bool(causal)), float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(q8.device))
    _check(code, "tts_attn_fwd_varlen_fp8")
    return out, lse


# The grouped-query calls are checked and made by a small native module (csrc/native.c): the
# calls of a decode step are shorter on the GPU than the same checks written here.
_nat = None


def _binding():
    """The native binding, given the library's entry points and torch's dtypes and streams."""
    global _nat
    if _nat is None:
        L = lib()
        try:
            from . import _native as m
        except ImportError as e:
            raise ImportError("the native binding is not built; run "
                              "tiled_top_sparse_gb300/_build.py") from e
        m.bind(tuple(ctypes.cast(f, ctypes.c_void_p).value
                     for f in (L.tts_rope_kv_append, L.tts_attn_decode_paged,
                               L.tts_attn_fwd_varlen_window)),
               (torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32),
               (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice,
                torch._C._cuda_setDevice))
        m.bind_more(tuple(ctypes.cast(f, ctypes.c_void_p).value
                          for f in (L.tts_rope_kv_append_axes, L.tts_attn_decode_tree,
                                    L.tts_kv_compact, L.tts_kv_fork, L.tts_qkv_rope_axes)),
                    torch.int64)
        _nat = m
    return _nat


def _attn_outputs(q, out, lse, want_lse, out_dtype):
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    return out, lse


def rope_kv_append(k, v, k_cache, v_cache, page_tables, past_lens, cu_new, max_new, k_scale=None,
                   v_scale=None, cos_sin=None, q=None, q_out=None, k_out=None, status=None,
                   want_k=False):
    """Append new tokens to a paged grouped-query cache, rotating q and k (tts_rope_kv_append).

    k, v bf16 [tokens, Hkv, d] and q [tokens, Hq, d] or None (views of a packed projection are
    taken as they are), caches [pages, Hkv, page_size, d] in bf16 or e4m3 codes (uint8 or
    float8_e4m3fn) with scales fp32 [pages, Hkv], page_tables int32 [batch, max_pages], past_lens
    int32 [batch], cu_new int32 [batch + 1], cos_sin of rope_cache or None (no rotation). The
    caches and scales are written in place. Returns (q_out bf16 [tokens, Hq, d] or None, k_out
    bf16 [tokens, Hkv, d]; k_out is None unless given or asked for with want_k)."""
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if want_k and k_out is None:
        k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
    code = (_nat or _binding()).rope_kv_append(k, v, k_cache, v_cache, page_tables, past_lens,
                                              cu_new, max_new, k_scale, v_scale, cos_sin, q, q_out,
                                              k_out, status)
    if code:
        raise TTSError(code, "tts_rope_kv_append")
    return q_out, k_out


def attn_decode_workspace_bytes(max_seqlen_q, num_heads_q, num_heads_kv, head_dim) -> int:
    return int(lib().tts_attn_decode_workspace_bytes(int(max_seqlen_q), int(num_heads_q),
                                                     int(num_heads_kv), int(head_dim)))


def attn_decode_paged(q, k_cache, v_cache, page_tables, kv_lens, scale, cu_seqlens_q=None,
                      max_seqlen_q=1, k_scale=None, v_scale=None, window=0, sinks=0, out=None,
                      lse=None, workspace=None, status=None, want_lse=True,
                      out_dtype=torch.float32):
    """Attention of each request's newest tokens over a paged grouped-query cache
    (tts_attn_decode_paged).

    q bf16 [tokens, Hq, d] (one token per request without cu_seqlens_q), the cache as in
    rope_kv_append, kv_lens int32 [batch] with the new tokens counted. window > 0: a token sees
    the last `window` positions up to its own and the first `sinks`. A workspace is allocated
    here when it is missing or too small. Returns (out [tokens, Hq, d] in out_dtype, or in out's
    dtype: fp32 or bf16; lse fp32 [tokens, Hq])."""
    out, lse = _attn_outputs(q, out, lse, want_lse, out_dtype)
    call = (_nat or _binding()).attn_decode_paged
    code = call(q, k_cache, v_cache, k_scale, v_scale, page_tables, kv_lens, cu_seqlens_q,
                max_seqlen_q, window, sinks, scale, out, lse, workspace, status)
    if code == TTS_ERR_WORKSPACE:  # missing or too small: nothing was enqueued
        with torch.cuda.device(q.device):
            need = attn_decode_workspace_bytes(max_seqlen_q, q.shape[1], k_cache.shape[1],
                                               q.shape[2])
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        code = call(q, k_cache, v_cache, k_scale, v_scale, page_tables, kv_lens, cu_seqlens_q,
                    max_seqlen_q, window, sinks, scale, out, lse, workspace, status)
    if code:
        raise TTSError(code, "tts_attn_decode_paged")
    return out, lse


def rope_axes(sections, interleaved=False) -> bytes:
    """The axis of every rotation pair (pair_axis of rope_kv_append_axes and qkv_rope_axes):
    sections[a] pairs turn by axis a. Consecutive runs, or, interleaved, pair j on axis j modulo
    their number as long as that one has pairs left, else on the first one that has."""
    sections = [int(n) for n in sections]
    _need(1 <= len(sections) <= 4 and min(sections) >= 0, "1 to 4 sections of 0 or more pairs")
    if not interleaved:
        return b"".join(bytes([a]) * n for a, n in enumerate(sections))
    axes, left, out = len(sections), list(sections), []
    for j in range(sum(sections)):
        a = j % axes if left[j % axes] > 0 else next(x for x in range(axes) if left[x] > 0)
        left[a] -= 1
        out.append(a)
    return bytes(out)


def rope_kv_append_axes(k, v, k_cache, v_cache, page_tables, past_lens, cu_new, max_new, positions,
                        pair_axis, cos_sin, k_scale=None, v_scale=None, q=None, q_out=None,
                        k_out=None, status=None, want_k=False):
    """rope_kv_append with explicit positions on one or several axes (tts_rope_kv_append_axes):
    positions int32 [axes, tokens], pair_axis bytes of head_dim/2 axes (rope_axes), cos_sin fp32
    [max_pos, head_dim/2, 2]. Images and video in a prompt, and drafted trees (one axis: the
    depth behind the cached tokens). Everything else, and what is returned, as there."""
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if want_k and k_out is None:
        k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=k.device)
    code = (_nat or _binding()).rope_kv_append_axes(
        k, v, k_cache, v_cache, page_tables, past_lens, cu_new, max_new, k_scale, v_scale, cos_sin,
        q, q_out, k_out, status, positions, pair_axis)
    if code:
        raise TTSError(code, "tts_rope_kv_append_axes")
    return q_out, k_out


def attn_decode_tree_workspace_bytes(max_seqlen_q, num_heads_q, num_heads_kv, head_dim) -> int:
    return int(lib().tts_attn_decode_tree_workspace_bytes(int(max_seqlen_q), int(num_heads_q),
                                                          int(num_heads_kv), int(head_dim)))


def attn_decode_tree(q, k_cache, v_cache, page_tables, kv_lens, tree_mask, scale, cu_seqlens_q=None,
                     max_seqlen_q=1, k_scale=None, v_scale=None, window=0, sinks=0, out=None,
                     lse=None, workspace=None, status=None, want_lse=True,
                     out_dtype=torch.float32):
    """Attention of a drafted tree's tokens over a paged grouped-query cache
    (tts_attn_decode_tree): as attn_decode_paged, but of its request's new tokens a token sees those
    of its mask. tree_mask int64 [tokens]: bit m, the request's new token m is seen (a tree's
    token has its ancestors' bits and its own)."""
    out, lse = _attn_outputs(q, out, lse, want_lse, out_dtype)
    call = (_nat or _binding()).attn_decode_tree
    code = call(q, k_cache, v_cache, k_scale, v_scale, page_tables, kv_lens, cu_seqlens_q,
                max_seqlen_q, window, sinks, scale, out, lse, workspace, status, tree_mask)
    if code == TTS_ERR_WORKSPACE:  # missing or too small: nothing was enqueued
        with torch.cuda.device(q.device):
            need = attn_decode_tree_workspace_bytes(max_seqlen_q, q.shape[1], k_cache.shape[1],
                                                    q.shape[2])
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        code = call(q, k_cache, v_cache, k_scale, v_scale, page_tables, kv_lens, cu_seqlens_q,
                    max_seqlen_q, window, sinks, scale, out, lse, workspace, status, tree_mask)
    if code:
        raise TTSError(code, "tts_attn_decode_tree")
    return out, lse


def kv_compact(k_cache, v_cache, page_tables, past_lens, path, path_lens, k_scale=None,
               v_scale=None, kv_lens=None, status=None):
    """Brings the accepted path of each request's drafted tree together in the cache
    (tts_kv_compact): of the new tokens behind past_lens[r] cached ones, path[r, :path_lens[r]]
    (int32 [batch, max_path], increasing, counted from 0) are kept, moved to the slots from
    past_lens[r] on. In place; returns kv_lens int32 [batch] = past_lens + path_lens."""
    if kv_lens is None:
        kv_lens = torch.empty_like(past_lens)
    code = (_nat or _binding()).kv_compact(k_cache, v_cache, page_tables, past_lens, path, path_lens,
                                          k_scale, v_scale, kv_lens, status)
    if code:
        raise TTSError(code, "tts_kv_compact")
    return kv_lens


def kv_fork(k_cache, v_cache, page_tables, kv_lens, parents, new_pages, k_scale=None, v_scale=None,
            tables_out=None, lens_out=None, status=None):
    """Requests that continue others' cached tokens (tts_kv_fork): new request i shares the full
    pages of request parents[i] (row of page_tables) and gets a copy of its last, partly filled
    page in new_pages[i] (int32, free pages; -1: the parent's row is taken as it is). Returns
    (tables int32 [children, max_pages], lengths int32 [children])."""
    if tables_out is None:
        tables_out = torch.empty((parents.numel(), page_tables.shape[1]), dtype=torch.int32,
                                 device=parents.device)
    if lens_out is None:
        lens_out = torch.empty(parents.numel(), dtype=torch.int32, device=parents.device)
    code = (_nat or _binding()).kv_fork(k_cache, v_cache, page_tables, kv_lens, parents, new_pages,
                                        k_scale, v_scale, tables_out, lens_out, status)
    if code:
        raise TTSError(code, "tts_kv_fork")
    return tables_out, lens_out


def qkv_rope_axes(x, w, bias, positions, pair_axis, cos_sin, num_heads, q=None, k=None, v=None,
                  status=None):
    """qkv_rope with positions on several axes (tts_qkv_rope_axes): positions int32 [axes, n] (row
    and column of a patch, time in front of them for video), pair_axis bytes of head_dim/2 axes
    (rope_axes), cos_sin fp32 [max_pos, d/2, 2] with each pair's own frequencies. Returns
    (q, k, v) bf16 [n, H, d]."""
    _need(isinstance(x, torch.Tensor) and x.dim() == 2 and w.dim() == 2 and int(num_heads) > 0,
          "x [n, hidden], w [3*H*d, hidden]")
    shape = (x.shape[0], int(num_heads), w.shape[0] // (3 * int(num_heads)))
    q, k, v = (torch.empty(shape, dtype=torch.bfloat16, device=x.device) if t is None else t
               for t in (q, k, v))
    try:
        call = (_nat or _binding()).qkv_rope_axes
    except ImportError:  # no binding: made from here, as qkv_rope is
        call = _qkv_rope_axes
    code = call(x, w, bias, positions, pair_axis, cos_sin, int(num_heads), q, k, v, status)
    if code:
        raise TTSError(code, "tts_qkv_rope_axes")
    return q, k, v


def _qkv_rope_axes(x, w, bias, positions, pair_axis, cos_sin, heads, q, k, v, status):
    """The binding's checks and call, on a machine that has none."""
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    for t, name, dtype in ((x, "x", bf16), (w, "w", bf16), (bias, "bias", f32),
                           (positions, "positions", i32), (cos_sin, "cos_sin", f32), (q, "q", bf16),
                           (k, "k", bf16), (v, "v", bf16), (status, "status", i32)):
        if t is None and name in ("bias", "status"):
            continue
        _cuda_contig(t, name, dtype)
        _need(t.device == x.device, f"{name} must be on x's device")
    n, hidden = x.shape
    _need(w.shape[0] > 0 and w.shape[0] % (3 * heads) == 0 and w.shape[1] == hidden,
          "x and w must be [n, hidden] and [3 * num_heads * head_dim, hidden]")
    d = w.shape[0] // (3 * heads)
    _need(bias is None or bias.numel() == w.shape[0], "bias must be [3 * num_heads * head_dim]")
    _need(cos_sin.dim() == 3 and cos_sin.shape[0] > 0 and tuple(cos_sin.shape[1:]) == (d // 2, 2),
          "cos_sin must be [max_pos, head_dim/2, 2] with a position at least")
    _need(positions.dim() == 2 and positions.shape[0] > 0 and positions.shape[1] == n,
          "positions must be [axes, tokens]")
    _need(isinstance(pair_axis, bytes) and len(pair_axis) == d // 2,
          "pair_axis must be bytes, one for each of the head_dim/2 pairs")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _need(tuple(t.shape) == (n, heads, d), f"{name} must be [n, num_heads, head_dim]")
    with torch.cuda.device(x.device):
        return lib().tts_qkv_rope_axes(
            _ptr(x), n, hidden, _ptr(w), _ptr(bias), _ptr(positions), positions.shape[0], pair_axis,
            _ptr(cos_sin), cos_sin.shape[0], heads, d, _ptr(q), _ptr(k), _ptr(v), _ptr(status),
            _stream(x.device))
