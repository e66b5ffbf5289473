"""libg2attn Python binding: Gemma 2 soft-capped local/global attention on B200.

Two layers:

* The C entry points under their own names (``g2attn_prefill``,
  ``g2attn_prefill_varlen``, ``g2attn_prefill_paged``, ``g2attn_decode_workspace_size``,
  ``g2attn_decode``, ``g2attn_decode_ring``, ``g2attn_decode_paged``,
  ``g2attn_decode_noalloc``, ``g2attn_backward_workspace_size``,
  ``g2attn_prefill_backward``, ``g2attn_varlen_backward_workspace_size``,
  ``g2attn_prefill_varlen_backward``, ``g2attn_rope``, ``g2attn_rope_append``,
  ``g2attn_rope_append_ring``, ``g2attn_rope_append_paged``,
  ``g2attn_extend_workspace_size``, ``g2attn_extend_paged``,
  ``g2attn_pages_workspace_size``, ``g2attn_pages_grow``,
  ``g2attn_pages_truncate``, ``g2attn_pages_fork``, ``g2attn_pages_compact``,
  ``g2attn_pages_copy``, ``g2attn_status_string``, ``g2attn_get_device_error``,
  ``g2attn_selftest_wait_timeout``): plain argument marshalling of integers,
  floats and raw pointers through ctypes, returning the status code.
* Tensor helpers (:func:`prefill`, :func:`prefill_varlen`, :func:`decode`,
  :func:`prefill_backward` and the others below)
  that take torch CUDA tensors, allocate the outputs with torch (memory
  plumbing only) and raise :class:`G2AttnError` on a nonzero status.

Every step of the attention runs in the CUDA kernels of ``libg2attn.so``.
There is no CPU or library fallback: if the shared library is missing the
first call raises.
"""
from __future__ import annotations

import ctypes
import decimal
import functools
import math
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libg2attn.so")

G2ATTN_OK = 0
G2ATTN_ERR_INVALID_ARG = 1
G2ATTN_ERR_UNSUPPORTED = 2
G2ATTN_ERR_MISALIGNED = 3
G2ATTN_ERR_CUDA = 4
G2ATTN_ERR_DEVICE_TIMEOUT = 5
G2ATTN_ERR_WORKSPACE = 6
G2ATTN_ERR_CACHE_LEN = 7
G2ATTN_ERR_CACHE_ROW = 8

EXPORTS = (
    "g2attn_prefill",
    "g2attn_prefill_varlen",
    "g2attn_prefill_paged",
    "g2attn_decode_workspace_size",
    "g2attn_decode",
    "g2attn_decode_ring",
    "g2attn_decode_paged",
    "g2attn_decode_noalloc",
    "g2attn_backward_workspace_size",
    "g2attn_prefill_backward",
    "g2attn_varlen_backward_workspace_size",
    "g2attn_prefill_varlen_backward",
    "g2attn_rope",
    "g2attn_rope_append",
    "g2attn_rope_append_ring",
    "g2attn_rope_append_paged",
    "g2attn_extend_workspace_size",
    "g2attn_extend_paged",
    "g2attn_pages_workspace_size",
    "g2attn_pages_grow",
    "g2attn_pages_truncate",
    "g2attn_pages_fork",
    "g2attn_pages_compact",
    "g2attn_pages_copy",
    "g2attn_status_string",
    "g2attn_get_device_error",
    "g2attn_selftest_wait_timeout",
)


class G2AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_name(status)} (status {status})")


_lib = None


def load_library():
    """Load libg2attn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"libg2attn.so is missing at {LIB_PATH}; build it with "
            "`python -m global_soft_capped_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.g2attn_prefill.argtypes = [P, P, P, P, P] + [I] * 7 + [F, F, I, P]
    lib.g2attn_prefill.restype = I
    lib.g2attn_prefill_varlen.argtypes = [P, P, P, P, P, P, P] + [I] * 8 + [F, F, I, P]
    lib.g2attn_prefill_varlen.restype = I
    lib.g2attn_prefill_paged.argtypes = [P, P, P, P, P, P, P, P] + [I] * 10 + [F, F, I, P]
    lib.g2attn_prefill_paged.restype = I
    lib.g2attn_decode_workspace_size.argtypes = [I, I, I, I]
    lib.g2attn_decode_workspace_size.restype = SZ
    lib.g2attn_decode.argtypes = [P, P, P, P, P, P] + [I] * 6 + [F, F, I, P, SZ, P]
    lib.g2attn_decode.restype = I
    lib.g2attn_decode_ring.argtypes = [P, P, P, P, P, P] + [I] * 6 + [F, F, I, P, SZ, P]
    lib.g2attn_decode_ring.restype = I
    lib.g2attn_decode_paged.argtypes = [P, P, P, P, P, P, P] + [I] * 8 + [F, F, I, P, SZ, P]
    lib.g2attn_decode_paged.restype = I
    lib.g2attn_decode_noalloc.argtypes = [P, P, P, P, P, P] + [I] * 6 + [F, F, I, P]
    lib.g2attn_decode_noalloc.restype = I
    lib.g2attn_backward_workspace_size.argtypes = [I, I, I]
    lib.g2attn_backward_workspace_size.restype = SZ
    lib.g2attn_prefill_backward.argtypes = [P] * 9 + [I] * 7 + [F, F, I, P, SZ, P]
    lib.g2attn_prefill_backward.restype = I
    lib.g2attn_varlen_backward_workspace_size.argtypes = [I, I, I]
    lib.g2attn_varlen_backward_workspace_size.restype = SZ
    lib.g2attn_prefill_varlen_backward.argtypes = [P] * 11 + [I] * 8 + [F, F, I, P, SZ, P]
    lib.g2attn_prefill_varlen_backward.restype = I
    LL = ctypes.c_longlong
    lib.g2attn_rope.argtypes = [P] * 6 + [I] * 6 + [F, I] + [LL] * 4 + [P]
    lib.g2attn_rope.restype = I
    lib.g2attn_rope_append.argtypes = [P] * 9 + [I] * 8 + [F] + [LL] * 3 + [P]
    lib.g2attn_rope_append.restype = I
    lib.g2attn_rope_append_ring.argtypes = [P] * 9 + [I] * 8 + [F] + [LL] * 3 + [P]
    lib.g2attn_rope_append_ring.restype = I
    lib.g2attn_rope_append_paged.argtypes = [P] * 10 + [I] * 10 + [F] + [LL] * 3 + [P]
    lib.g2attn_rope_append_paged.restype = I
    lib.g2attn_extend_workspace_size.argtypes = [I, I]
    lib.g2attn_extend_workspace_size.restype = SZ
    lib.g2attn_extend_paged.argtypes = [P] * 8 + [I] * 9 + [F, F, I, P, SZ, P]
    lib.g2attn_extend_paged.restype = I
    lib.g2attn_pages_workspace_size.argtypes = [I, I]
    lib.g2attn_pages_workspace_size.restype = SZ
    lib.g2attn_pages_grow.argtypes = [P] * 7 + [I] * 4 + [P, SZ, P]
    lib.g2attn_pages_grow.restype = I
    lib.g2attn_pages_truncate.argtypes = [P] * 4 + [I] * 4 + [P]
    lib.g2attn_pages_truncate.restype = I
    lib.g2attn_pages_fork.argtypes = [P] * 9 + [I] * 4 + [P, SZ, P]
    lib.g2attn_pages_fork.restype = I
    lib.g2attn_pages_compact.argtypes = [P] * 5 + [I] * 3 + [P, SZ, P]
    lib.g2attn_pages_compact.restype = I
    lib.g2attn_pages_copy.argtypes = [P, I, P, P, I, I, SZ, P]
    lib.g2attn_pages_copy.restype = I
    lib.g2attn_status_string.argtypes = [I]
    lib.g2attn_status_string.restype = ctypes.c_char_p
    lib.g2attn_get_device_error.argtypes = []
    lib.g2attn_get_device_error.restype = I
    lib.g2attn_selftest_wait_timeout.argtypes = [I]
    lib.g2attn_selftest_wait_timeout.restype = I
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# C entry points, same names and argument order as include/g2attn.h
# ---------------------------------------------------------------------------
def g2attn_prefill(q, k, v, out, lse, B, T, S, H, Hkv, d, q_offset, query_scale, softcap,
                   window, stream):
    return load_library().g2attn_prefill(q, k, v, out, lse, B, T, S, H, Hkv, d, q_offset,
                                         query_scale, softcap, window, stream)


def g2attn_prefill_varlen(q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q,
                          total_k, max_T, max_S, H, Hkv, d, query_scale, softcap, window, stream):
    return load_library().g2attn_prefill_varlen(q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k,
                                                num_seqs, total_q, total_k, max_T, max_S, H, Hkv,
                                                d, query_scale, softcap, window, stream)


def g2attn_prefill_paged(q, k_blocks, v_blocks, out, lse, cu_seqlens_q, block_table, seq_lens_k,
                         num_seqs, total_q, num_blocks, block_size, max_blocks_per_seq, max_T,
                         max_S, H, Hkv, d, query_scale, softcap, window, stream):
    return load_library().g2attn_prefill_paged(q, k_blocks, v_blocks, out, lse, cu_seqlens_q,
                                               block_table, seq_lens_k, num_seqs, total_q,
                                               num_blocks, block_size, max_blocks_per_seq, max_T,
                                               max_S, H, Hkv, d, query_scale, softcap, window,
                                               stream)


def g2attn_backward_workspace_size(B, T, H):
    return load_library().g2attn_backward_workspace_size(B, T, H)


def g2attn_prefill_backward(q, k, v, out, lse, dout, dq, dk, dv, B, T, S, H, Hkv, d, q_offset,
                            query_scale, softcap, window, workspace, workspace_bytes, stream):
    return load_library().g2attn_prefill_backward(q, k, v, out, lse, dout, dq, dk, dv, B, T, S,
                                                  H, Hkv, d, q_offset, query_scale, softcap,
                                                  window, workspace, workspace_bytes, stream)


def g2attn_varlen_backward_workspace_size(num_seqs, total_q, H):
    return load_library().g2attn_varlen_backward_workspace_size(num_seqs, total_q, H)


def g2attn_prefill_varlen_backward(q, k, v, out, lse, dout, dq, dk, dv, cu_seqlens_q,
                                   cu_seqlens_k, num_seqs, total_q, total_k, max_T, max_S, H,
                                   Hkv, d, query_scale, softcap, window, workspace,
                                   workspace_bytes, stream):
    return load_library().g2attn_prefill_varlen_backward(
        q, k, v, out, lse, dout, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, num_seqs, total_q,
        total_k, max_T, max_S, H, Hkv, d, query_scale, softcap, window, workspace,
        workspace_bytes, stream)


def g2attn_decode_workspace_size(num_seqs, H, d, max_cache_len):
    return load_library().g2attn_decode_workspace_size(num_seqs, H, d, max_cache_len)


def g2attn_decode(q, k_cache, v_cache, cu_seqlens_k, out, lse, num_seqs, total_k, max_cache_len,
                  H, Hkv, d, query_scale, softcap, window, workspace, workspace_bytes, stream):
    return load_library().g2attn_decode(q, k_cache, v_cache, cu_seqlens_k, out, lse, num_seqs,
                                        total_k, max_cache_len, H, Hkv, d, query_scale, softcap,
                                        window, workspace, workspace_bytes, stream)


def g2attn_decode_ring(q, k_ring, v_ring, seq_lens, out, lse, num_seqs, ring_size, max_cache_len,
                       H, Hkv, d, query_scale, softcap, window, workspace, workspace_bytes,
                       stream):
    return load_library().g2attn_decode_ring(q, k_ring, v_ring, seq_lens, out, lse, num_seqs,
                                             ring_size, max_cache_len, H, Hkv, d, query_scale,
                                             softcap, window, workspace, workspace_bytes, stream)


def g2attn_decode_paged(q, k_blocks, v_blocks, block_table, seq_lens, out, lse, num_seqs,
                        num_blocks, block_size, max_blocks_per_seq, max_cache_len, H, Hkv, d,
                        query_scale, softcap, window, workspace, workspace_bytes, stream):
    return load_library().g2attn_decode_paged(q, k_blocks, v_blocks, block_table, seq_lens, out,
                                              lse, num_seqs, num_blocks, block_size,
                                              max_blocks_per_seq, max_cache_len, H, Hkv, d,
                                              query_scale, softcap, window, workspace,
                                              workspace_bytes, stream)


def g2attn_decode_noalloc(q, k_cache, v_cache, cu_seqlens_k, out, lse, num_seqs, total_k,
                          max_cache_len, H, Hkv, d, query_scale, softcap, window, stream):
    """Decode with the library's static scratch instead of a caller workspace,
    for callers that cannot allocate device memory at call time."""
    return load_library().g2attn_decode_noalloc(q, k_cache, v_cache, cu_seqlens_k, out, lse,
                                                num_seqs, total_k, max_cache_len, H, Hkv, d,
                                                query_scale, softcap, window, stream)


def g2attn_rope(q, k, q_out, k_out, positions, freqs, num_tokens, H, Hkv, d, rotary_dim,
                interleaved, mscale, inverse, q_stride, k_stride, q_out_stride, k_out_stride,
                stream):
    return load_library().g2attn_rope(q, k, q_out, k_out, positions, freqs, num_tokens, H, Hkv,
                                      d, rotary_dim, interleaved, mscale, inverse, q_stride,
                                      k_stride, q_out_stride, k_out_stride, stream)


def g2attn_rope_append(q, k, v, q_out, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, freqs,
                       num_seqs, total_q, total_k, H, Hkv, d, rotary_dim, interleaved, mscale,
                       q_stride, k_stride, v_stride, stream):
    return load_library().g2attn_rope_append(q, k, v, q_out, k_cache, v_cache, cu_seqlens_q,
                                             cu_seqlens_k, freqs, num_seqs, total_q, total_k, H,
                                             Hkv, d, rotary_dim, interleaved, mscale, q_stride,
                                             k_stride, v_stride, stream)


def g2attn_rope_append_ring(q, k, v, q_out, k_ring, v_ring, cu_seqlens_q, seq_lens, freqs,
                            num_seqs, total_q, ring_size, H, Hkv, d, rotary_dim, interleaved,
                            mscale, q_stride, k_stride, v_stride, stream):
    return load_library().g2attn_rope_append_ring(q, k, v, q_out, k_ring, v_ring, cu_seqlens_q,
                                                  seq_lens, freqs, num_seqs, total_q, ring_size,
                                                  H, Hkv, d, rotary_dim, interleaved, mscale,
                                                  q_stride, k_stride, v_stride, stream)


def g2attn_rope_append_paged(q, k, v, q_out, k_blocks, v_blocks, cu_seqlens_q, block_table,
                             seq_lens, freqs, num_seqs, total_q, num_blocks, block_size,
                             max_blocks_per_seq, H, Hkv, d, rotary_dim, interleaved, mscale,
                             q_stride, k_stride, v_stride, stream):
    return load_library().g2attn_rope_append_paged(q, k, v, q_out, k_blocks, v_blocks,
                                                   cu_seqlens_q, block_table, seq_lens, freqs,
                                                   num_seqs, total_q, num_blocks, block_size,
                                                   max_blocks_per_seq, H, Hkv, d, rotary_dim,
                                                   interleaved, mscale, q_stride, k_stride,
                                                   v_stride, stream)


def g2attn_extend_workspace_size(max_T, d):
    return load_library().g2attn_extend_workspace_size(max_T, d)


def g2attn_extend_paged(q, k_blocks, v_blocks, out, lse, cu_seqlens_q, block_table, seq_lens,
                        num_seqs, total_q, num_blocks, block_size, max_blocks_per_seq, max_T, H,
                        Hkv, d, query_scale, softcap, window, workspace, workspace_bytes, stream):
    return load_library().g2attn_extend_paged(q, k_blocks, v_blocks, out, lse, cu_seqlens_q,
                                              block_table, seq_lens, num_seqs, total_q,
                                              num_blocks, block_size, max_blocks_per_seq, max_T,
                                              H, Hkv, d, query_scale, softcap, window, workspace,
                                              workspace_bytes, stream)


def g2attn_pages_workspace_size(num_seqs, num_blocks):
    return load_library().g2attn_pages_workspace_size(num_seqs, num_blocks)


def g2attn_pages_grow(block_table, seq_lens, ref_counts, add, granted, copy_src, copy_dst,
                      num_seqs, num_blocks, block_size, max_blocks_per_seq, workspace,
                      workspace_bytes, stream):
    return load_library().g2attn_pages_grow(block_table, seq_lens, ref_counts, add, granted,
                                            copy_src, copy_dst, num_seqs, num_blocks, block_size,
                                            max_blocks_per_seq, workspace, workspace_bytes,
                                            stream)


def g2attn_pages_truncate(block_table, seq_lens, ref_counts, keep, num_seqs, num_blocks,
                          block_size, max_blocks_per_seq, stream):
    return load_library().g2attn_pages_truncate(block_table, seq_lens, ref_counts, keep, num_seqs,
                                                num_blocks, block_size, max_blocks_per_seq,
                                                stream)


def g2attn_pages_fork(block_table, seq_lens, parents, new_table, new_lens, ref_counts, copy_src,
                      copy_dst, granted, num_seqs, num_blocks, block_size, max_blocks_per_seq,
                      workspace, workspace_bytes, stream):
    return load_library().g2attn_pages_fork(block_table, seq_lens, parents, new_table, new_lens,
                                            ref_counts, copy_src, copy_dst, granted, num_seqs,
                                            num_blocks, block_size, max_blocks_per_seq, workspace,
                                            workspace_bytes, stream)


def g2attn_pages_compact(block_table, ref_counts, copy_src, copy_dst, num_live, num_seqs,
                         num_blocks, max_blocks_per_seq, workspace, workspace_bytes, stream):
    return load_library().g2attn_pages_compact(block_table, ref_counts, copy_src, copy_dst,
                                               num_live, num_seqs, num_blocks, max_blocks_per_seq,
                                               workspace, workspace_bytes, stream)


def g2attn_pages_copy(caches, num_caches, src, dst, num_pairs, num_blocks, page_bytes, stream):
    return load_library().g2attn_pages_copy(caches, num_caches, src, dst, num_pairs, num_blocks,
                                            page_bytes, stream)


def g2attn_status_string(status):
    return load_library().g2attn_status_string(status).decode()


def g2attn_get_device_error():
    return load_library().g2attn_get_device_error()


def g2attn_selftest_wait_timeout(timeout_us):
    return load_library().g2attn_selftest_wait_timeout(timeout_us)


def status_name(status: int) -> str:
    try:
        return g2attn_status_string(status)
    except Exception:  # library not loadable: still give a readable message
        return f"status {status}"


# ---------------------------------------------------------------------------
# Tensor helpers (torch allocates; the kernels compute)
# ---------------------------------------------------------------------------
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check_bf16(*ts):
    import torch
    for t in ts:
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("expected contiguous bf16 CUDA tensors")


def prefill(q, k, v, *, q_offset=0, query_scale=1.0, softcap=50.0, window=0, out=None,
            lse=None, want_lse=True, stream=None):
    """Dense prefill. q (B,T,H,d), k/v (B,S,Hkv,d) -> (out (B,T,H,d), lse (B,H,T) | None)."""
    import torch
    _check_bf16(q, k, v)
    B, T, H, d = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    st = g2attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, T, S, H, Hkv, d,
                        int(q_offset), float(query_scale), float(softcap), int(window),
                        _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_prefill")
    return out, lse


def prefill_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_T, max_S, *, query_scale=1.0,
                   softcap=50.0, window=0, out=None, lse=None, want_lse=True, stream=None):
    """Packed prefill. q (sum T,H,d), k/v (sum S,Hkv,d); cu_seqlens int32 CUDA tensors."""
    import torch
    _check_bf16(q, k, v)
    total_q, H, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    num_seqs = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    st = g2attn_prefill_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                               _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), num_seqs, total_q, total_k,
                               int(max_T), int(max_S), H, Hkv, d, float(query_scale),
                               float(softcap), int(window), _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_prefill_varlen")
    return out, lse


def backward_workspace(B, T, H, device="cuda"):
    """A device buffer of g2attn_backward_workspace_size(B, T, H) bytes."""
    import torch
    n = g2attn_backward_workspace_size(B, T, H)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def prefill_backward(q, k, v, out, lse, dout, *, q_offset=0, query_scale=1.0, softcap=50.0,
                     window=0, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients of :func:`prefill`: returns (dq, dk, dv) like q, k, v (bf16)."""
    import torch
    _check_bf16(q, k, v, out, dout)
    B, T, H, d = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = backward_workspace(B, T, H, q.device)
    st = g2attn_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, T, S, H, Hkv, d, int(q_offset),
                                 float(query_scale), float(softcap), int(window), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_prefill_backward")
    return dq, dk, dv


def prefill_varlen_backward(q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_T, max_S,
                            *, query_scale=1.0, softcap=50.0, window=0, workspace=None, dq=None,
                            dk=None, dv=None, stream=None):
    """Gradients of :func:`prefill_varlen`: returns (dq, dk, dv), packed like q, k, v."""
    import torch
    _check_bf16(q, k, v, out, dout)
    total_q, H, d = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    num_seqs = cu_seqlens_q.numel() - 1
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        n = g2attn_varlen_backward_workspace_size(num_seqs, total_q, H)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    st = g2attn_prefill_varlen_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
        _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), num_seqs, total_q, total_k,
        int(max_T), int(max_S), H, Hkv, d, float(query_scale), float(softcap), int(window),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_prefill_varlen_backward")
    return dq, dk, dv


def decode_workspace(num_seqs, H, d, max_cache_len, device="cuda"):
    import torch
    nbytes = g2attn_decode_workspace_size(num_seqs, H, d, max_cache_len)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def decode(q, k_cache, v_cache, cu_seqlens_k, max_cache_len, *, query_scale=1.0, softcap=50.0,
           window=0, out=None, lse=None, workspace=None, want_lse=True, stream=None):
    """Decode. q (n,H,d), caches (sum L,Hkv,d), cu_seqlens_k int32 CUDA (n+1)."""
    import torch
    _check_bf16(q, k_cache, v_cache)
    n, H, d = q.shape
    total_k, Hkv = k_cache.shape[0], k_cache.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((n, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(n, H, d, max_cache_len, q.device)
    st = g2attn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cu_seqlens_k), _ptr(out),
                       _ptr(lse), n, total_k, int(max_cache_len), H, Hkv, d, float(query_scale),
                       float(softcap), int(window), _ptr(workspace), workspace.numel(),
                       _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_decode")
    return out, lse


def decode_ring(q, k_ring, v_ring, seq_lens, window, max_cache_len=None, *, query_scale=1.0,
                softcap=50.0, out=None, lse=None, workspace=None, want_lse=True, stream=None):
    """Decode over ring caches (n, R, Hkv, d); seq_lens int32 CUDA (n,)."""
    import torch
    _check_bf16(q, k_ring, v_ring)
    n, H, d = q.shape
    R, Hkv = k_ring.shape[1], k_ring.shape[2]
    max_cache_len = int(window if max_cache_len is None else max_cache_len)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((n, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(n, H, d, max_cache_len, q.device)
    st = g2attn_decode_ring(_ptr(q), _ptr(k_ring), _ptr(v_ring), _ptr(seq_lens), _ptr(out),
                            _ptr(lse), n, R, max_cache_len, H, Hkv, d, float(query_scale),
                            float(softcap), int(window), _ptr(workspace), workspace.numel(),
                            _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_decode_ring")
    return out, lse


def decode_paged(q, k_blocks, v_blocks, block_table, seq_lens, max_cache_len, *,
                 query_scale=1.0, softcap=50.0, window=0, out=None, lse=None, workspace=None,
                 want_lse=True, stream=None):
    """Decode over paged caches (num_blocks, bs, Hkv, d); block_table int32 (n, max_blocks)."""
    import torch
    _check_bf16(q, k_blocks, v_blocks)
    n, H, d = q.shape
    nb, bs, Hkv = k_blocks.shape[0], k_blocks.shape[1], k_blocks.shape[2]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((n, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = decode_workspace(n, H, d, max_cache_len, q.device)
    st = g2attn_decode_paged(_ptr(q), _ptr(k_blocks), _ptr(v_blocks), _ptr(block_table),
                             _ptr(seq_lens), _ptr(out), _ptr(lse), n, nb, bs,
                             block_table.shape[1], int(max_cache_len), H, Hkv, d,
                             float(query_scale), float(softcap), int(window), _ptr(workspace),
                             workspace.numel(), _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_decode_paged")
    return out, lse


def prefill_paged(q, k_blocks, v_blocks, cu_seqlens_q, block_table, seq_lens_k, max_T, max_S, *,
                  query_scale=1.0, softcap=50.0, window=0, out=None, lse=None, want_lse=True,
                  stream=None):
    """Chunked prefill: packed q (sum T,H,d) over paged K/V (num_blocks, bs, Hkv, d)."""
    import torch
    _check_bf16(q, k_blocks, v_blocks)
    total_q, H, d = q.shape
    nb, bs, Hkv = k_blocks.shape[0], k_blocks.shape[1], k_blocks.shape[2]
    num_seqs = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    st = g2attn_prefill_paged(_ptr(q), _ptr(k_blocks), _ptr(v_blocks), _ptr(out), _ptr(lse),
                              _ptr(cu_seqlens_q), _ptr(block_table), _ptr(seq_lens_k), num_seqs,
                              total_q, nb, bs, block_table.shape[1], int(max_T), int(max_S), H,
                              Hkv, d, float(query_scale), float(softcap), int(window),
                              _stream(stream))
    if st != G2ATTN_OK:
        raise G2AttnError(st, "g2attn_prefill_paged")
    return out, lse


# ---------------------------------------------------------------------------
# Rotary positions, cache appends, chunk attention, pages
# ---------------------------------------------------------------------------
class RopePlan(NamedTuple):
    """What the rotary calls need besides the tensors: made once by :func:`rope_plan`."""
    freqs: object        # int64 CUDA tensor (rotary_dim / 2): turns per position * 2^64
    rotary_dim: int
    interleaved: bool = False
    mscale: float = 1.0


# Digits that the tables are made with: 64-bit fixed point of a turn per position
# wants 20, and what positions of 31 bits multiply must be right behind them.
_DIGITS = decimal.Context(prec=60)
_TWO_PI = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def _rope_radians(rotary_dim, base=10000.0, scaling=None, factor=1.0, trained_len=8192,
                  fast_turns=32.0, slow_turns=1.0):
    """:func:`rope_frequencies` in decimal numbers of 60 digits."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    rotary_dim = int(rotary_dim)  # (of a numpy integer, too)
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    half, mscale = rotary_dim // 2, 1.0
    num = decimal.Decimal
    with decimal.localcontext(_DIGITS):
        wide, times = num(float(base)), num(float(factor))
        if scaling == "ntk" and rotary_dim > 2:
            wide *= times ** (num(rotary_dim) / (rotary_dim - 2))
        inv = [wide ** (num(-2 * i) / rotary_dim) for i in range(half)]
        if scaling == "linear":
            inv = [w / times for w in inv]
        elif scaling == "yarn":
            def pair(turns):  # the (fractional) pair that turns so often over trained_len
                return (rotary_dim * math.log(trained_len / (turns * 2.0 * math.pi))
                        / (2.0 * math.log(base)))
            low = max(math.floor(pair(fast_turns)), 0)
            high = min(math.ceil(pair(slow_turns)), rotary_dim - 1)
            ramp = [min(max(num(i - low) / max(num(high - low), num("0.001")), num(0)), num(1))
                    for i in range(half)]
            inv = [w / times * r + w * (1 - r) for w, r in zip(inv, ramp)]
            mscale = 0.1 * math.log(factor) + 1.0
    return inv, mscale


def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, trained_len=8192,
                     fast_turns=32.0, slow_turns=1.0):
    """Radians per position of every pair, and the factor on the rotation.

    w_i = base^(-2 i / rotary_dim), then for a context ``factor`` times the
    trained one, ``scaling``: None; "linear", w_i / factor; "ntk", the base times
    factor^(rotary_dim / (rotary_dim - 2)); "yarn", w_i / factor for pairs that
    turn less than ``slow_turns`` times over ``trained_len`` positions, w_i for
    those that turn more than ``fast_turns`` times, a ramp between, and the
    rotation times 0.1 ln(factor) + 1.
    """
    inv, mscale = _rope_radians(rotary_dim, base, scaling, factor, trained_len, fast_turns,
                                slow_turns)
    return [float(w) for w in inv], mscale


def rope_plan(rotary_dim, *, interleaved=False, device="cuda", frequencies=None, mscale=None,
              **scaling):
    """A :class:`RopePlan` on ``device`` from the arguments of
    :func:`rope_frequencies` (``scaling``), or from ``frequencies`` (radians per
    position, as doubles). The table holds their turns per position rounded once,
    to 2^-65: phases of any int32 position are right to 2^-34 turns."""
    if torch is None:
        _load_torch()
    m = 1.0
    if frequencies is None:
        frequencies, m = _rope_radians(rotary_dim, **scaling)
    elif scaling:
        raise ValueError("give frequencies or their parameters, not both")
    else:
        frequencies = [decimal.Decimal(float(w)) for w in frequencies]
    if len(frequencies) != rotary_dim // 2:
        raise ValueError("one frequency per pair")
    with decimal.localcontext(_DIGITS):
        turns = [int((w / _TWO_PI * 2 ** 64).to_integral_value()) % 2 ** 64 for w in frequencies]
    freqs = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64,
                         device=device)
    return RopePlan(freqs, int(rotary_dim), bool(interleaved), m if mscale is None else mscale)


def _load_torch():
    """torch for the helpers below, imported with the first of them (a call of
    these takes a few microseconds, and an import statement in each of the
    functions it runs through is a good part of that)."""
    global torch, _raw_stream, _current_device
    import torch as t
    _raw_stream, _current_device = t._C._cuda_getCurrentRawStream, t._C._cuda_getDevice
    torch = t


torch = None


def _launch(name, device, stream, args):
    """Calls a C entry point with ``args`` and the stream, its device current."""
    index = device.index
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    fn = getattr(_lib or load_library(), name)
    if _current_device() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st != G2ATTN_OK:
        raise G2AttnError(st, name)


def _heads(name, t, device=None):
    """(token count, heads, d, elements between tokens) of a (..., heads, d)
    bf16 CUDA tensor whose tokens are evenly spaced and whose heads are dense."""
    if torch is None:
        _load_torch()
    if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() not in (3, 4):
        raise ValueError(f"{name}: expected a bf16 CUDA tensor (tokens, heads, d) or (B, T, heads, d)")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on another device than the first tensor")
    sh, st = t.shape, t.stride()
    H, d = sh[-2], sh[-1]
    n, step = sh[-3], st[-3]
    if t.dim() == 4:
        if sh[0] > 1 and n > 1 and st[0] != n * step:
            raise ValueError(f"{name}: the tokens of the batch are not evenly spaced")
        if n == 1:
            step = st[0]
        n *= sh[0]
    if n == 1:
        step = H * d
    if st[-1] != 1 or (H > 1 and st[-2] != d):
        raise ValueError(f"{name}: heads of a token must be dense")
    return n, H, d, step


def _new(stream, make, *args, **kwargs):
    """A tensor for a call on ``stream``, from that stream's memory when one is
    given: memory of the current stream may still be in use by its earlier work,
    which the call does not wait for. The current stream, where the result is
    most likely read, is recorded as a user of it."""
    if stream is None:
        return make(*args, **kwargs)
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make(*args, **kwargs)
    t.record_stream(here)
    return t


def _workspace(t, device):
    """(pointer, bytes) of a caller's workspace."""
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _dense_like(t):
    """A new packed tensor of a shape that :func:`_heads` accepted: evenly spaced
    tokens, for which empty_like's layout is the packed one in the same order."""
    o = torch.empty_like(t)
    return o if o.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _ints(name, t, n, device, dtype=None):
    if dtype is None:
        dtype = torch.int32
    if (t.dtype != dtype or t.device != device or not t.is_contiguous()
            or (n is not None and t.numel() != n)):
        raise ValueError(f"{name}: expected {'' if n is None else n} contiguous {dtype} values "
                         f"on {device}")
    return t.data_ptr()


def _cache(name, t, dims, Hkv, d, device):
    """Pointer of a contiguous bf16 cache (..., Hkv, d)."""
    sh = t.shape
    if (t.dtype != torch.bfloat16 or t.device != device or len(sh) != dims or sh[-1] != d
            or sh[-2] != Hkv or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous bf16 tensor of {dims} dimensions on "
                         f"{device} that ends in (Hkv, d)")
    return t.data_ptr()


def _like_cache(name, t, other):
    if (t.dtype != other.dtype or t.device != other.device or t.shape != other.shape
            or not t.is_contiguous()):
        raise ValueError(f"{name}: expected a tensor like the K cache")
    return t.data_ptr()


def _plan_args(plan, device):
    return _ints("plan.freqs", plan.freqs, plan.rotary_dim // 2, device, torch.int64)


def _rope(q, k, positions, plan, inverse, out, stream):
    n, H, d, qs = _heads("q", q)
    nk, Hkv, dk, ks = _heads("k", k, q.device)
    if nk != n or dk != d:
        raise ValueError("q and k differ in tokens or head size")
    if out is None:
        qo, ko = _new(stream, _dense_like, q), _new(stream, _dense_like, k)
        qos, kos = H * d, Hkv * d
    else:
        qo, ko = out
        if qo.shape != q.shape or ko.shape != k.shape:
            raise ValueError("out: expected the shapes of q and k")
        qos, kos = _heads("out q", qo, q.device)[3], _heads("out k", ko, q.device)[3]
    _launch("g2attn_rope", q.device, stream, (
        q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(),
        _ints("positions", positions, n, q.device), _plan_args(plan, q.device), n, H, Hkv, d,
        plan.rotary_dim, int(plan.interleaved), plan.mscale, inverse, qs, ks, qos, kos))
    return qo, ko


def rope(q, k, positions, plan, *, out=None, stream=None):
    """Rotary positions: q (B,T,H,d) or (tokens,H,d), k alike with Hkv, either
    of them a slice of a fused projection; positions int32 CUDA, one per token.
    Returns rotated (q, k); ``out=(q, k)`` rotates in place."""
    return _rope(q, k, positions, plan, 0, out, stream)


def rope_backward(dq, dk, positions, plan, *, out=None, stream=None):
    """Gradients of :func:`rope`: of its results in, of its inputs out."""
    return _rope(dq, dk, positions, plan, 1, out, stream)


def _append(q, k, v, cu_seqlens_q, num_seqs, q_out, stream):
    """Checks common to the appends: (sizes, strides, q_out, cu pointer)."""
    n, H, d, qs = _heads("q", q)
    nk, Hkv, dk, ks = _heads("k", k, q.device)
    nv, Hv, dv, vs = _heads("v", v, q.device)
    if (nk, dk) != (n, d) or (nv, Hv, dv) != (n, Hkv, d):
        raise ValueError("q, k and v differ in tokens, heads or head size")
    if q_out is None:
        q_out = _new(stream, _dense_like, q)
    elif q_out.shape != q.shape or not q_out.is_contiguous() or q_out.dtype != q.dtype \
            or q_out.device != q.device:
        raise ValueError("q_out: expected a contiguous bf16 tensor like q")
    cu = None
    if cu_seqlens_q is not None:
        cu = _ints("cu_seqlens_q", cu_seqlens_q, num_seqs + 1, q.device)
    elif n != num_seqs:
        raise ValueError("without cu_seqlens_q every sequence has one token")
    return n, H, Hkv, d, qs, ks, vs, q_out, cu


def rope_append(q, k, v, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, plan, *, q_out=None,
                stream=None):
    """Rotates q (returned) and k and writes k and v to the last rows of every
    sequence of a packed cache (sum L,Hkv,d); cu_seqlens_q None: one token each.
    The lengths are those with the new tokens (with an older one the tokens
    would overwrite the sequence's last rows)."""
    n_seqs = cu_seqlens_k.numel() - 1
    n, H, Hkv, d, qs, ks, vs, q_out, cu = _append(q, k, v, cu_seqlens_q, n_seqs, q_out, stream)
    kc, vc = _cache("k_cache", k_cache, 3, Hkv, d, q.device), _like_cache("v_cache", v_cache, k_cache)
    _launch("g2attn_rope_append", q.device, stream, (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), kc, vc, cu,
        _ints("cu_seqlens_k", cu_seqlens_k, None, q.device), _plan_args(plan, q.device), n_seqs, n,
        k_cache.shape[0], H, Hkv, d, plan.rotary_dim, int(plan.interleaved), plan.mscale, qs, ks,
        vs))
    return q_out


def rope_append_ring(q, k, v, k_ring, v_ring, cu_seqlens_q, seq_lens, plan, *, q_out=None,
                     stream=None):
    """:func:`rope_append` into ring caches (n,R,Hkv,d); seq_lens with the new tokens."""
    n_seqs = seq_lens.numel()
    n, H, Hkv, d, qs, ks, vs, q_out, cu = _append(q, k, v, cu_seqlens_q, n_seqs, q_out, stream)
    kc, vc = _cache("k_ring", k_ring, 4, Hkv, d, q.device), _like_cache("v_ring", v_ring, k_ring)
    if k_ring.shape[0] != n_seqs:
        raise ValueError("k_ring: expected one ring per sequence")
    _launch("g2attn_rope_append_ring", q.device, stream, (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), kc, vc, cu,
        _ints("seq_lens", seq_lens, None, q.device), _plan_args(plan, q.device), n_seqs, n,
        k_ring.shape[1], H, Hkv, d, plan.rotary_dim, int(plan.interleaved), plan.mscale, qs, ks,
        vs))
    return q_out


def rope_append_paged(q, k, v, k_blocks, v_blocks, cu_seqlens_q, block_table, seq_lens, plan, *,
                      q_out=None, stream=None):
    """:func:`rope_append` into paged caches (num_blocks,bs,Hkv,d); block_table
    int32 (n, max_blocks), seq_lens with the new tokens."""
    n_seqs = seq_lens.numel()
    n, H, Hkv, d, qs, ks, vs, q_out, cu = _append(q, k, v, cu_seqlens_q, n_seqs, q_out, stream)
    kc = _cache("k_blocks", k_blocks, 4, Hkv, d, q.device)
    vc = _like_cache("v_blocks", v_blocks, k_blocks)
    if block_table.dim() != 2 or block_table.shape[0] != n_seqs:
        raise ValueError("block_table: expected one row per sequence")
    _launch("g2attn_rope_append_paged", q.device, stream, (
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), kc, vc, cu,
        _ints("block_table", block_table, None, q.device),
        _ints("seq_lens", seq_lens, None, q.device), _plan_args(plan, q.device), n_seqs, n,
        k_blocks.shape[0], k_blocks.shape[1], block_table.shape[1], H, Hkv, d, plan.rotary_dim,
        int(plan.interleaved), plan.mscale, qs, ks, vs))
    return q_out


@functools.lru_cache(maxsize=256)
def _extend_bytes(max_T, d):
    """Workspace bytes; a size function, so the call (a microsecond) is made once."""
    return load_library().g2attn_extend_workspace_size(max_T, d)


@functools.lru_cache(maxsize=256)
def _pages_bytes(num_seqs, num_blocks):
    return load_library().g2attn_pages_workspace_size(num_seqs, num_blocks)


def extend_workspace(max_T, d, device="cuda"):
    """A device buffer of g2attn_extend_workspace_size(max_T, d) bytes."""
    if torch is None:
        _load_torch()
    return torch.empty(max(g2attn_extend_workspace_size(max_T, d), 16), dtype=torch.uint8,
                       device=device)


def extend_paged(q, k_blocks, v_blocks, cu_seqlens_q, block_table, seq_lens, max_T, *,
                 query_scale=1.0, softcap=50.0, window=0, out=None, lse=None, workspace=None,
                 want_lse=True, stream=None):
    """Attention of short chunks of new tokens, packed q (sum T,H,d), over paged
    caches (num_blocks,bs,Hkv,d) that already hold them; seq_lens with the new
    tokens. Returns (out (sum T,H,d), lse (H, sum T) | None)."""
    if torch is None:
        _load_torch()
    if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q: expected a contiguous bf16 CUDA tensor (tokens, H, d)")
    total_q, H, d = q.shape
    max_T = int(max_T)
    kc = _cache("k_blocks", k_blocks, 4, k_blocks.shape[-2], d, q.device)
    vc = _like_cache("v_blocks", v_blocks, k_blocks)
    n = seq_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("block_table: expected one row per sequence")
    if out is None:
        out = _new(stream, torch.empty_like, q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device \
            or not out.is_contiguous():
        raise ValueError("out: expected a contiguous bf16 tensor like q")
    if lse is None and want_lse:
        lse = _new(stream, q.new_empty, (H, total_q), dtype=torch.float32)
    elif lse is not None and (lse.shape != (H, total_q) or lse.dtype != torch.float32
                              or lse.device != q.device or not lse.is_contiguous()):
        raise ValueError("lse: expected a contiguous fp32 tensor (H, tokens)")
    if workspace is None:
        workspace = _new(stream, q.new_empty, _extend_bytes(max_T, d), dtype=torch.uint8)
    ws, ws_bytes = _workspace(workspace, q.device)
    _launch("g2attn_extend_paged", q.device, stream, (
        q.data_ptr(), kc, vc, out.data_ptr(), None if lse is None else lse.data_ptr(),
        _ints("cu_seqlens_q", cu_seqlens_q, n + 1, q.device),
        _ints("block_table", block_table, None, q.device),
        _ints("seq_lens", seq_lens, None, q.device), n, total_q, k_blocks.shape[0],
        k_blocks.shape[1], block_table.shape[1], max_T, H, k_blocks.shape[2], d, query_scale,
        softcap, int(window), ws, ws_bytes))
    return out, lse


def pages_workspace(num_seqs, num_blocks, device="cuda"):
    """A device buffer of g2attn_pages_workspace_size(num_seqs, num_blocks) bytes."""
    if torch is None:
        _load_torch()
    return torch.empty(max(g2attn_pages_workspace_size(num_seqs, num_blocks), 16),
                       dtype=torch.uint8, device=device)


def _pages_ws(workspace, stream, block_table, num_seqs, num_blocks):
    """The workspace (kept alive by the caller), its pointer and bytes."""
    if workspace is None:
        workspace = _new(stream, block_table.new_empty,
                         (_pages_bytes(num_seqs, num_blocks) + 3) // 4)
    return workspace, *_workspace(workspace, block_table.device)


def _table(block_table, ref_counts):
    """(pointer, sequences, columns, pages, counts' pointer) of a page state."""
    if torch is None:
        _load_torch()
    if not block_table.is_cuda or block_table.dim() != 2:
        raise ValueError("block_table: expected an int32 CUDA tensor (num_seqs, max_blocks)")
    dev = block_table.device
    return (_ints("block_table", block_table, None, dev), block_table.shape[0],
            block_table.shape[1], ref_counts.numel(), _ints("ref_counts", ref_counts, None, dev))


def pages_grow(block_table, seq_lens, ref_counts, add, block_size, *, copies=False,
               workspace=None, stream=None):
    """Lengthens every sequence by add rows with fresh pages, in place; returns
    granted (num_seqs,) int32, 0 where the pages ran out. A sequence that was cut
    (:func:`pages_truncate`) inside a page which a fork shares needs a copy of it:
    with ``copies`` the result is (granted, copy_src, copy_dst) for
    :func:`pages_copy`, without it such a sequence is refused. Each of several
    sequences that share such a page and grow in one call gets a copy. Issue the
    copies before the next grow, fork or compact, and not together with theirs:
    the pages read may count as free by now. A refused sequence keeps its length:
    give the appends none of its tokens, they would overwrite its last rows."""
    tp, n, cols, nb, rp = _table(block_table, ref_counts)
    dev = block_table.device
    ws, wp, wb = _pages_ws(workspace, stream, block_table, n, nb)
    src = dst = None
    if copies:
        granted, src, dst = _new(stream, block_table.new_empty, (3, n)).unbind(0)
    else:
        granted = _new(stream, block_table.new_empty, n)
    _launch("g2attn_pages_grow", dev, stream, (
        tp, _ints("seq_lens", seq_lens, n, dev), rp, _ints("add", add, n, dev), granted.data_ptr(),
        None if src is None else src.data_ptr(), None if dst is None else dst.data_ptr(), n, nb,
        int(block_size), cols, wp, wb))
    return (granted, src, dst) if copies else granted


def pages_truncate(block_table, seq_lens, ref_counts, keep, block_size, *, stream=None):
    """Cuts every sequence to at most keep rows and gives its pages back, in place."""
    tp, n, cols, nb, rp = _table(block_table, ref_counts)
    dev = block_table.device
    _launch("g2attn_pages_truncate", dev, stream, (
        tp, _ints("seq_lens", seq_lens, n, dev), rp, _ints("keep", keep, n, dev), n, nb,
        int(block_size), cols))


def pages_fork(block_table, seq_lens, ref_counts, parents, block_size, *, workspace=None,
               stream=None):
    """Every sequence s a fork of sequence parents[s] (s: stays). ref_counts in
    place; returns (block_table, seq_lens, copy_src, copy_dst, granted), the
    first two new. Copy the pages (:func:`pages_copy`) before appending and before
    the next grow, fork or compact, as those of :func:`pages_grow`."""
    tp, n, cols, nb, rp = _table(block_table, ref_counts)
    dev = block_table.device
    table = _new(stream, torch.empty_like, block_table)
    lens, src, dst, granted = _new(stream, block_table.new_empty, (4, n)).unbind(0)
    ws, wp, wb = _pages_ws(workspace, stream, block_table, n, nb)
    _launch("g2attn_pages_fork", dev, stream, (
        tp, _ints("seq_lens", seq_lens, n, dev), _ints("parents", parents, n, dev),
        table.data_ptr(), lens.data_ptr(), rp, src.data_ptr(), dst.data_ptr(), granted.data_ptr(),
        n, nb, int(block_size), cols, wp, wb))
    return table, lens, src, dst, granted


def pages_compact(block_table, ref_counts, *, workspace=None, stream=None):
    """Renumbers the live pages to the front of the cache, in place; returns
    (copy_src, copy_dst, num_live) for :func:`pages_copy`, to be issued before
    anything reads the caches and before the next grow, fork or compact."""
    tp, n, cols, nb, rp = _table(block_table, ref_counts)
    dev = block_table.device
    src, dst = _new(stream, block_table.new_empty, (2, nb // 2)).unbind(0)
    live = _new(stream, block_table.new_empty, 1)
    ws, wp, wb = _pages_ws(workspace, stream, block_table, n, nb)
    _launch("g2attn_pages_compact", dev, stream, (
        tp, rp, src.data_ptr(), dst.data_ptr(), live.data_ptr(), n, nb, cols, wp, wb))
    return src, dst, live


def pages_copy(caches, src, dst, *, stream=None):
    """Copies pages src to pages dst in every cache (num_blocks, ...) of a list
    (K and V of all layers), all of one shape and type."""
    if torch is None:
        _load_torch()
    caches = list(caches)
    if not caches or caches[0].numel() == 0:
        raise ValueError("caches: expected at least one tensor with pages")
    first = caches[0]
    dev, shape, kind, n = first.device, first.shape, first.dtype, src.numel()
    for c in caches:
        if not c.is_cuda or c.device != dev or c.shape != shape or c.dtype != kind \
                or not c.is_contiguous():
            raise ValueError("caches: expected contiguous CUDA tensors of one shape and type")
    sp, dp = _ints("src", src, None, dev), _ints("dst", dst, n, dev)
    if n == 0:
        return
    ptrs = (ctypes.c_void_p * len(caches))(*[c.data_ptr() for c in caches])
    _launch("g2attn_pages_copy", dev, stream, (
        ptrs, len(caches), sp, dp, n, shape[0],
        first.numel() // shape[0] * first.element_size()))
