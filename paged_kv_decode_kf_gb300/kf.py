"""Thin ctypes binding of the C-ABI library (include/kf.h), same names.

Argument marshalling only: every step of the decode path runs in the
library's CUDA kernels. Tensors must be CUDA tensors in the layouts kf.h
states; the current torch stream is used unless one is given. Importing this
module loads ``_lib/libkf.so`` and fails loudly if it has not been built
(``__graft_entry__.build()``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libkf.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("the kf CUDA library is not built (%s missing); run "
                      "`python -c 'import __graft_entry__ as g; g.build()'`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

KF_OK, KF_ERR_INVALID, KF_ERR_UNSUPPORTED, KF_ERR_CUDA, KF_ERR_DEVICE = range(5)
KF_BF16, KF_F32 = 0, 1
KF_SPLITS_BALANCED = 0  # num_splits of the step calls: balanced one-wave schedule
KF_DEVERR_BLOCK_ID = 0x01
KF_DEVERR_CONTEXT_LEN = 0x02
KF_DEVERR_MAX_CONTEXT = 0x04
KF_DEVERR_APPEND_POS = 0x08
KF_DEVERR_TIMEOUT = 0x10
KF_DEVERR_RANGE = 0x20

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float

_lib.kf_append_kv.restype = _i32
_lib.kf_append_kv.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i64, _vp]
_lib.kf_paged_decode_attention.restype = _i32
_lib.kf_paged_decode_attention.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                           _i32, _i32, _i64, _f32, _i32, _vp, _vp, _vp]
_lib.kf_choose_num_splits.restype = _i32
_lib.kf_choose_num_splits.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _vp, _i32]
_lib.kf_choose_num_splits_for.restype = _i32
_lib.kf_choose_num_splits_for.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _vp, _i32]
_lib.kf_choose_num_splits_fp8.restype = _i32
_lib.kf_choose_num_splits_fp8.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _vp, _i32]
_lib.kf_paged_multiquery_attention.restype = _i32
_lib.kf_paged_multiquery_attention.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                               _i32, _i32, _i32, _i32, _i64, _f32, _i32, _vp, _vp, _vp]
_lib.kf_merge_partials.restype = _i32
_lib.kf_merge_partials.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _vp]
_lib.kf_decode_step_workspace_size.restype = ctypes.c_size_t
_lib.kf_decode_step_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.kf_decode_step.restype = _i32
_lib.kf_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                _i32, _i64, _f32, _i32, _vp, ctypes.c_size_t, _vp, _i32, _vp, _vp]
_lib.kf_decode_step_static.restype = _i32
_lib.kf_decode_step_merge_partials.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                                _i32, _i32, _i64, _f32, _i32, _vp, _vp, _i32, _vp,
                                                ctypes.c_size_t, _vp, _i32, _vp, _vp]
_lib.kf_decode_step_merge_partials.restype = _i32
_lib.kf_decode_step_static.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                       _i32, _i32, _i64, _f32, _i32, _vp, _i32, _vp, _vp]
KF_STATIC_SCRATCH_BYTES = 32 * 1024 * 1024
_lib.kf_append_kv_fp8.restype = _i32
_lib.kf_append_kv_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i64, _vp]
_lib.kf_paged_decode_attention_fp8.restype = _i32
_lib.kf_paged_decode_attention_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                               _i32, _i32, _i32, _i64, _f32, _i32, _vp, _vp, _vp]
_lib.kf_decode_step_fp8.restype = _i32
_lib.kf_decode_step_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                    _i32, _i32, _i32, _i64, _f32, _i32, _vp, ctypes.c_size_t, _vp, _i32, _vp,
                                    _vp]
_sz = ctypes.c_size_t
_lib.kf_append_latent.restype = _i32
_lib.kf_append_latent.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i64, _vp]
_lib.kf_latent_workspace_size.restype = _sz
_lib.kf_latent_workspace_size.argtypes = [_i32] * 4
_lib.kf_latent_attention.restype = _i32
_lib.kf_latent_attention.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                     _i32, _i32, _i64, _f32, _vp, _sz, _vp, _i32, _vp, _vp]
_lib.kf_latent_expanded_workspace_size.restype = _sz
_lib.kf_latent_expanded_workspace_size.argtypes = [_i32] * 6
_lib.kf_latent_attention_expanded.restype = _i32
_lib.kf_latent_attention_expanded.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                              _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64, _f32, _vp, _sz, _vp,
                                              _i32, _vp, _vp]
_lib.kf_accumulate_attention.restype = _i32
_lib.kf_accumulate_attention.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                         _i32, _i32, _i64, _f32, _vp, _vp, _vp, _i64, _vp]
_lib.kf_accumulate_attention_fp8.restype = _i32
_lib.kf_accumulate_attention_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                             _i32, _i32, _i32, _i32, _i64, _f32, _vp, _vp, _vp, _i64, _vp]
_lib.kf_evict_workspace_size.restype = _sz
_lib.kf_evict_workspace_size.argtypes = [_i32] * 3
_lib.kf_evict_tokens.restype = _i32
_lib.kf_evict_tokens.argtypes = [_vp, _vp, _i64, _vp, _i32, _vp, _i32, _i32, _i32, _i64, _vp, _vp, _i64, _vp, _vp,
                                 _vp, _i32, _i32, _i32, _vp, _vp, _sz, _vp]
_lib.kf_get_device_error.restype = _i32
_lib.kf_check_bounded_wait.restype = _i32
_lib.kf_check_bounded_wait.argtypes = [_vp]
_lib.kf_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), _vp]
_lib.kf_status_string.restype = ctypes.c_char_p
_lib.kf_status_string.argtypes = [_i32]
_lib.kf_version.restype = _i32
_lib.kf_version.argtypes = []


class KfError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, _lib.kf_status_string(status).decode(), status))


def raw():
    """The loaded ctypes library (for callers that pass raw pointers)."""
    return _lib


def _check(status: int, what: str) -> None:
    if status != KF_OK:
        raise KfError(status, what)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _io(t: torch.Tensor, dtype, name: str) -> int:
    """A per-step input or output of the kf_decode_step calls: a CUDA tensor, or
    a pinned host tensor the GPU reads or writes in place (zero-copy)."""
    if not t.is_cuda and not t.is_pinned():
        raise ValueError("%s must be a CUDA tensor or pinned host memory" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def kf_version() -> int:
    return _lib.kf_version()


def kf_append_kv(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, block_tables: torch.Tensor,
                 context_lens_before: torch.Tensor, stream=None) -> None:
    """Write each request's new K/V row at position context_lens_before[b]."""
    nb, bs, hkv, d = k_cache.shape
    B = block_tables.shape[0]
    _check(_lib.kf_append_kv(
        _dev(k_new, torch.bfloat16, "k_new"), _dev(v_new, torch.bfloat16, "v_new"),
        _dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
        _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
        _dev(context_lens_before, torch.int32, "context_lens_before"), B, hkv, d, bs, nb,
        _stream(stream)), "kf_append_kv")


def kf_choose_num_splits(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                         block_size: int, max_context_len: int, context_lens_host=None,
                         device: Optional[int] = None, num_sms: Optional[int] = None,
                         kv_dtype: str = "bf16") -> int:
    """The library's split count for this batch (host-side plan)."""
    arr = None
    ptr = None
    if context_lens_host is not None:
        arr = torch.as_tensor(context_lens_host, dtype=torch.int32).cpu().contiguous()
        ptr = arr.data_ptr()
    if kv_dtype == "fp8":
        if num_sms is None:
            dev = torch.cuda.current_device() if device is None else device
            num_sms = torch.cuda.get_device_properties(dev).multi_processor_count
        n = _lib.kf_choose_num_splits_fp8(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                          max_context_len, ptr, num_sms)
    elif num_sms is not None:
        n = _lib.kf_choose_num_splits_for(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                          max_context_len, ptr, num_sms)
    else:
        dev = torch.cuda.current_device() if device is None else device
        n = _lib.kf_choose_num_splits(batch, num_q_heads, num_kv_heads, head_dim, block_size,
                                      max_context_len, ptr, dev)
    if n < 1:
        raise KfError(KF_ERR_INVALID, "kf_choose_num_splits")
    return n


def kf_paged_decode_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_tables: torch.Tensor, context_lens: torch.Tensor,
                              max_context_len: int, scale: float, num_splits: int,
                              out_partial: Optional[torch.Tensor] = None,
                              lse_partial: Optional[torch.Tensor] = None,
                              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Split-KV decode attention; returns (out_partial [S,B,Hq,D], lse_partial [S,B,Hq])."""
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if out_partial is None:
        out_partial = torch.empty((num_splits, B, hq, d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((num_splits, B, hq), dtype=torch.float32, device=q.device)
    _check(_lib.kf_paged_decode_attention(
        _dev(q, torch.bfloat16, "q"), _dev(k_cache, torch.bfloat16, "k_cache"),
        _dev(v_cache, torch.bfloat16, "v_cache"), _dev(block_tables, torch.int32, "block_tables"),
        block_tables.shape[1], _dev(context_lens, torch.int32, "context_lens"), int(max_context_len),
        B, hq, hkv, d, bs, nb, float(scale), int(num_splits),
        _dev(out_partial, torch.float32, "out_partial"), _dev(lse_partial, torch.float32, "lse_partial"),
        _stream(stream)), "kf_paged_decode_attention")
    return out_partial, lse_partial


def kf_paged_multiquery_attention(q: torch.Tensor, q_start: torch.Tensor, k_cache: torch.Tensor,
                                  v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  causal: bool, max_context_len: int, max_query_len: int, scale: float,
                                  num_splits: int, out_partial: Optional[torch.Tensor] = None,
                                  lse_partial: Optional[torch.Tensor] = None,
                                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Multi-query paged attention (chunked prefill / shared prefix); returns
    (out_partial [S, Nq, Hq, D], lse_partial [S, Nq, Hq])."""
    Nq, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    B = block_tables.shape[0]
    if out_partial is None:
        out_partial = torch.empty((num_splits, Nq, hq, d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((num_splits, Nq, hq), dtype=torch.float32, device=q.device)
    _check(_lib.kf_paged_multiquery_attention(
        _dev(q, torch.bfloat16, "q"), _dev(q_start, torch.int32, "q_start"),
        _dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
        _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), int(bool(causal)), int(max_context_len),
        int(max_query_len), B, Nq, hq, hkv, d, bs, nb, float(scale), int(num_splits),
        _dev(out_partial, torch.float32, "out_partial"), _dev(lse_partial, torch.float32, "lse_partial"),
        _stream(stream)), "kf_paged_multiquery_attention")
    return out_partial, lse_partial


def kf_merge_partials(out_partial: torch.Tensor, lse_partial: torch.Tensor,
                      out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                      lse_out: Optional[torch.Tensor] = None, want_lse: bool = True,
                      stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """LSE merge of [S,B,Hq,D]/[S,B,Hq] partials; returns (out [B,Hq,D], lse [B,Hq] or None)."""
    S, B, hq, d = out_partial.shape
    if out is None:
        out = torch.empty((B, hq, d), dtype=out_dtype, device=out_partial.device)
    code = {torch.float32: KF_F32, torch.bfloat16: KF_BF16}.get(out.dtype)
    if code is None:
        raise ValueError("out must be float32 or bfloat16")
    if lse_out is None and want_lse:
        lse_out = torch.empty((B, hq), dtype=torch.float32, device=out_partial.device)
    _check(_lib.kf_merge_partials(
        _dev(out_partial, torch.float32, "out_partial"), _dev(lse_partial, torch.float32, "lse_partial"),
        S, B, hq, d, _dev(out, out.dtype, "out"), code,
        None if lse_out is None else _dev(lse_out, torch.float32, "lse_out"), _stream(stream)),
        "kf_merge_partials")
    return out, lse_out


def kf_decode_step_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                  num_splits: int) -> int:
    return int(_lib.kf_decode_step_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, num_splits))


def make_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, num_splits: int,
                   device=None) -> torch.Tensor:
    """A zero-filled workspace for kf_decode_step (the zero fill is required once)."""
    n = kf_decode_step_workspace_size(batch, num_q_heads, num_kv_heads, head_dim, num_splits)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def kf_decode_step(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, block_tables: torch.Tensor, context_lens_before: torch.Tensor,
                   max_context_len: int, scale: float, num_splits: int,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype=torch.float32, lse_out: Optional[torch.Tensor] = None, want_lse: bool = True,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Append + split attention + merge in one launch; returns (out, lse).
    q, k_new, v_new, block_tables, context_lens_before, out and lse_out may be
    pinned host tensors (read and written by the kernel in place)."""
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if out is None:
        out = torch.empty((B, hq, d), dtype=out_dtype, device=k_cache.device)
    code = {torch.float32: KF_F32, torch.bfloat16: KF_BF16}.get(out.dtype)
    if code is None:
        raise ValueError("out must be float32 or bfloat16")
    if lse_out is None and want_lse:
        lse_out = torch.empty((B, hq), dtype=torch.float32, device=k_cache.device)
    if workspace is None and num_splits != 1:
        raise ValueError("num_splits > 1 and the balanced schedule need a workspace (make_workspace)")
    ws_ptr = None if workspace is None else _dev(workspace, torch.uint8, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check(_lib.kf_decode_step(
        _io(q, torch.bfloat16, "q"), _io(k_new, torch.bfloat16, "k_new"), _io(v_new, torch.bfloat16, "v_new"),
        _dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
        _io(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
        _io(context_lens_before, torch.int32, "context_lens_before"), int(max_context_len), B, hq, hkv, d,
        bs, nb, float(scale), int(num_splits), ws_ptr, ws_bytes, _io(out, out.dtype, "out"), code,
        None if lse_out is None else _io(lse_out, torch.float32, "lse_out"), _stream(stream)),
        "kf_decode_step")
    return out, lse_out


def kf_decode_step_merge_partials(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                                  k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                                  context_lens_before: torch.Tensor, max_context_len: int, scale: float,
                                  num_splits: int, extra_out_partial: torch.Tensor,
                                  extra_lse_partial: torch.Tensor, workspace: torch.Tensor,
                                  out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                                  lse_out: Optional[torch.Tensor] = None, want_lse: bool = True,
                                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """kf_decode_step whose merge also takes the extra partials
    ([n, B, Hq, D] and [n, B, Hq]); returns (out, lse)."""
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    n_ex = int(extra_lse_partial.shape[0])
    if tuple(extra_out_partial.shape) != (n_ex, B, hq, d) or tuple(extra_lse_partial.shape) != (n_ex, B, hq):
        raise ValueError("extra partials must be [n, B, Hq, D] and [n, B, Hq]")
    if out is None:
        out = torch.empty((B, hq, d), dtype=out_dtype, device=k_cache.device)
    code = {torch.float32: KF_F32, torch.bfloat16: KF_BF16}.get(out.dtype)
    if code is None:
        raise ValueError("out must be float32 or bfloat16")
    if lse_out is None and want_lse:
        lse_out = torch.empty((B, hq), dtype=torch.float32, device=k_cache.device)
    _check(_lib.kf_decode_step_merge_partials(
        _io(q, torch.bfloat16, "q"), _io(k_new, torch.bfloat16, "k_new"), _io(v_new, torch.bfloat16, "v_new"),
        _dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
        _io(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
        _io(context_lens_before, torch.int32, "context_lens_before"), int(max_context_len), B, hq, hkv, d,
        bs, nb, float(scale), int(num_splits), _dev(extra_out_partial, torch.float32, "extra_out_partial"),
        _dev(extra_lse_partial, torch.float32, "extra_lse_partial"), n_ex,
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _io(out, out.dtype, "out"), code,
        None if lse_out is None else _io(lse_out, torch.float32, "lse_out"), _stream(stream)),
        "kf_decode_step_merge_partials")
    return out, lse_out


def kf_decode_step_static(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                          k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                          context_lens_before: torch.Tensor, max_context_len: int, scale: float,
                          num_splits: int, out: torch.Tensor, lse_out: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """kf_decode_step with the library's own fixed scratch instead of a workspace,
    for callers that may not allocate device memory; `out` (and `lse_out`) must
    be given. Calls on one device must not overlap on the GPU."""
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    code = {torch.float32: KF_F32, torch.bfloat16: KF_BF16}.get(out.dtype)
    if code is None:
        raise ValueError("out must be float32 or bfloat16")
    _check(_lib.kf_decode_step_static(
        _io(q, torch.bfloat16, "q"), _io(k_new, torch.bfloat16, "k_new"), _io(v_new, torch.bfloat16, "v_new"),
        _dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
        _io(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
        _io(context_lens_before, torch.int32, "context_lens_before"), int(max_context_len), B, hq, hkv, d,
        bs, nb, float(scale), int(num_splits), _io(out, out.dtype, "out"), code,
        None if lse_out is None else _io(lse_out, torch.float32, "lse_out"), _stream(stream)),
        "kf_decode_step_static")


def _dev8(t: torch.Tensor, name: str) -> int:
    """An FP8 E4M3 cache: uint8 codes or torch.float8_e4m3fn."""
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError("%s must be uint8 E4M3 codes or float8_e4m3fn, got %s" % (name, t.dtype))
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % name)
    return t.data_ptr()


def kf_append_kv_fp8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                     context_lens_before, stream=None) -> None:
    """Quantise and write each request's new K/V row into E4M3 caches."""
    nb, bs, hkv, d = k_cache.shape
    B = block_tables.shape[0]
    _check(_lib.kf_append_kv_fp8(
        _dev(k_new, torch.bfloat16, "k_new"), _dev(v_new, torch.bfloat16, "v_new"),
        _dev8(k_cache, "k_cache"), _dev8(v_cache, "v_cache"), _dev(k_scale, torch.float32, "k_scale"),
        _dev(v_scale, torch.float32, "v_scale"), _dev(block_tables, torch.int32, "block_tables"),
        block_tables.shape[1], _dev(context_lens_before, torch.int32, "context_lens_before"), B, hkv, d,
        bs, nb, _stream(stream)), "kf_append_kv_fp8")


def kf_paged_decode_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                  max_context_len: int, scale: float, num_splits: int,
                                  out_partial=None, lse_partial=None, stream=None):
    """Split-KV decode attention over E4M3 caches; returns (out_partial, lse_partial)."""
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if out_partial is None:
        out_partial = torch.empty((num_splits, B, hq, d), dtype=torch.float32, device=q.device)
    if lse_partial is None:
        lse_partial = torch.empty((num_splits, B, hq), dtype=torch.float32, device=q.device)
    _check(_lib.kf_paged_decode_attention_fp8(
        _dev(q, torch.bfloat16, "q"), _dev8(k_cache, "k_cache"), _dev8(v_cache, "v_cache"),
        _dev(k_scale, torch.float32, "k_scale"), _dev(v_scale, torch.float32, "v_scale"),
        _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
        _dev(context_lens, torch.int32, "context_lens"), int(max_context_len), B, hq, hkv, d, bs, nb,
        float(scale), int(num_splits), _dev(out_partial, torch.float32, "out_partial"),
        _dev(lse_partial, torch.float32, "lse_partial"), _stream(stream)), "kf_paged_decode_attention_fp8")
    return out_partial, lse_partial


def kf_decode_step_fp8(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                       context_lens_before, max_context_len: int, scale: float, num_splits: int,
                       workspace=None, out=None, out_dtype=torch.float32, lse_out=None, want_lse=True,
                       stream=None):
    """Single-launch decode step over E4M3 caches; returns (out, lse). The
    per-step tensors may be pinned host memory, as for kf_decode_step."""
    B, hq, d = q.shape
    nb, bs, hkv, d2 = k_cache.shape
    if out is None:
        out = torch.empty((B, hq, d), dtype=out_dtype, device=k_cache.device)
    code = {torch.float32: KF_F32, torch.bfloat16: KF_BF16}.get(out.dtype)
    if code is None:
        raise ValueError("out must be float32 or bfloat16")
    if lse_out is None and want_lse:
        lse_out = torch.empty((B, hq), dtype=torch.float32, device=k_cache.device)
    if workspace is None and num_splits != 1:
        raise ValueError("num_splits > 1 and the balanced schedule need a workspace (make_workspace)")
    _check(_lib.kf_decode_step_fp8(
        _io(q, torch.bfloat16, "q"), _io(k_new, torch.bfloat16, "k_new"), _io(v_new, torch.bfloat16, "v_new"),
        _dev8(k_cache, "k_cache"), _dev8(v_cache, "v_cache"), _dev(k_scale, torch.float32, "k_scale"),
        _dev(v_scale, torch.float32, "v_scale"), _io(block_tables, torch.int32, "block_tables"),
        block_tables.shape[1], _io(context_lens_before, torch.int32, "context_lens_before"),
        int(max_context_len), B, hq, hkv, d, bs, nb, float(scale), int(num_splits),
        None if workspace is None else _dev(workspace, torch.uint8, "workspace"),
        0 if workspace is None else workspace.numel(), _io(out, out.dtype, "out"), code,
        None if lse_out is None else _io(lse_out, torch.float32, "lse_out"), _stream(stream)),
        "kf_decode_step_fp8")
    return out, lse_out


def _latent_dims(latent_cache: torch.Tensor) -> Tuple[int, int, int]:
    """(num_blocks, block_size, latent_dim) of a latent cache."""
    shape = latent_cache.shape
    if len(shape) != 3 or shape[2] <= KF_ROPE_DIM:
        raise ValueError("latent_cache must be [num_blocks, block_size, latent_dim + %d]" % KF_ROPE_DIM)
    return shape[0], shape[1], shape[2] - KF_ROPE_DIM


def _shape(t: torch.Tensor, shape, name: str) -> None:
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))


# The current stream's handle of a device; the public call builds a Stream object
# first, several microseconds on a slow host core.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(name: str, index: int, stream, *args) -> None:
    """Call the library's `name` with device `index` current and the stream
    appended to the arguments."""
    if index < 0:
        raise ValueError("all tensors must be CUDA tensors")
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _call(name, index, stream, *args)
    handle = _raw_stream(index) if stream is None and _raw_stream is not None else _stream(stream)
    status = getattr(_lib, name)(*args, handle)
    if status != KF_OK:
        raise KfError(status, name)


def _on(index: int, t: torch.Tensor, dtype, name: str) -> int:
    """The address of a contiguous tensor of `dtype` on device `index`."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != index:
        raise ValueError("%s must be on the call's device, cuda:%d, got %s" % (name, index, t.device))
    return _dev(t, dtype, name)   # names what is wrong


KF_ROPE_DIM = 64  # width of the rotary part of a latent row


def kf_append_latent(latent_new: torch.Tensor, latent_cache: torch.Tensor, block_tables: torch.Tensor,
                     context_lens_before: torch.Tensor, row_start: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Write each request's new latent rows (one, or rows row_start[b]..row_start[b+1]-1)
    from position context_lens_before[b] on."""
    nb, bs, r = _latent_dims(latent_cache)
    B, columns = block_tables.shape
    n = latent_new.shape[0]
    _shape(latent_new, (n, r + KF_ROPE_DIM), "latent_new")
    _shape(context_lens_before, (B,), "context_lens_before")
    if row_start is not None:
        _shape(row_start, (B + 1,), "row_start")
    elif n != B:
        raise ValueError("latent_new must hold one row a request without row_start")
    dev = latent_cache.get_device()
    _call("kf_append_latent", dev, stream,
          _on(dev, latent_new, torch.bfloat16, "latent_new"),
          None if row_start is None else _on(dev, row_start, torch.int32, "row_start"),
          _on(dev, latent_cache, torch.bfloat16, "latent_cache"), _on(dev, block_tables, torch.int32, "block_tables"),
          columns, _on(dev, context_lens_before, torch.int32, "context_lens_before"), B, n, r, KF_ROPE_DIM, bs, nb)


def kf_latent_workspace_size(batch: int, max_query_len: int, num_heads: int, latent_dim: int) -> int:
    return int(_lib.kf_latent_workspace_size(batch, max_query_len, num_heads, latent_dim))


def make_latent_workspace(batch: int, max_query_len: int, num_heads: int, latent_dim: int,
                          device=None) -> torch.Tensor:
    """A workspace for kf_latent_attention (any contents)."""
    dev = torch.device(device or "cuda")
    with torch.cuda.device(dev):
        n = kf_latent_workspace_size(batch, max_query_len, num_heads, latent_dim)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=dev)


def _latent_call(q, width, out_width, B, context_lens, q_start, out, out_dtype, lse_out, want_lse):
    """Shape checks and outputs shared by the two forms; returns (num_q_tokens,
    num_heads, out, out code, lse_out)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != width:
        raise ValueError("q must be [num_q_tokens, num_heads, %d], got %s" % (width, list(shape)))
    nq, h, _ = shape
    if context_lens.shape != (B,):
        _shape(context_lens, (B,), "context_lens")
    if q_start is not None:
        if q_start.shape != (B + 1,):
            _shape(q_start, (B + 1,), "q_start")
    elif nq != B:
        raise ValueError("q must hold one query token a request without q_start")
    if out is None:
        out = torch.empty((nq, h, out_width), dtype=out_dtype, device=q.device)
    elif out.shape != (nq, h, out_width):
        _shape(out, (nq, h, out_width), "out")
    dtype = out.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise ValueError("out must be float32 or bfloat16")
    if lse_out is None:
        if want_lse:
            lse_out = torch.empty((nq, h), dtype=torch.float32, device=q.device)
    elif lse_out.shape != (nq, h):
        _shape(lse_out, (nq, h), "lse_out")
    return nq, h, out, KF_F32 if dtype is torch.float32 else KF_BF16, lse_out


def kf_latent_attention(q: torch.Tensor, latent_cache: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, max_context_len: int, scale: float, workspace: torch.Tensor,
                        q_start: Optional[torch.Tensor] = None, max_query_len: int = 1, causal: bool = True,
                        out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                        lse_out: Optional[torch.Tensor] = None, want_lse: bool = True,
                        stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Latent attention, absorbed form: q [Nq, H, R + 64] over the latent cache;
    returns (out [Nq, H, R], lse [Nq, H])."""
    nb, bs, r = _latent_dims(latent_cache)
    B, columns = block_tables.shape
    nq, h, out, code, lse_out = _latent_call(q, r + KF_ROPE_DIM, r, B, context_lens, q_start, out, out_dtype, lse_out,
                                             want_lse)
    dev = q.get_device()
    _call("kf_latent_attention", dev, stream,
          _on(dev, q, torch.bfloat16, "q"), None if q_start is None else _on(dev, q_start, torch.int32, "q_start"),
          _on(dev, latent_cache, torch.bfloat16, "latent_cache"), _on(dev, block_tables, torch.int32, "block_tables"),
          columns, _on(dev, context_lens, torch.int32, "context_lens"), 1 if causal else 0,
          int(max_context_len), int(max_query_len), B, nq, h, r, KF_ROPE_DIM, bs, nb, float(scale),
          _on(dev, workspace, torch.uint8, "workspace"), workspace.numel(), _on(dev, out, out.dtype, "out"), code,
          None if lse_out is None else _on(dev, lse_out, torch.float32, "lse_out"))
    return out, lse_out


def kf_latent_expanded_workspace_size(batch: int, num_q_tokens: int, max_context_len: int, num_heads: int,
                                      nope_dim: int, v_dim: int) -> int:
    return int(_lib.kf_latent_expanded_workspace_size(batch, num_q_tokens, max_context_len, num_heads, nope_dim,
                                                      v_dim))


def make_latent_expanded_workspace(batch: int, num_q_tokens: int, max_context_len: int, num_heads: int,
                                   nope_dim: int, v_dim: int, device=None) -> torch.Tensor:
    """A workspace for kf_latent_attention_expanded (any contents)."""
    n = kf_latent_expanded_workspace_size(batch, num_q_tokens, max_context_len, num_heads, nope_dim, v_dim)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def kf_latent_attention_expanded(q: torch.Tensor, latent_cache: torch.Tensor, w_uk: torch.Tensor,
                                 w_uv: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                                 max_context_len: int, scale: float, workspace: torch.Tensor,
                                 q_start: Optional[torch.Tensor] = None, max_query_len: int = 1,
                                 causal: bool = True, out: Optional[torch.Tensor] = None,
                                 out_dtype=torch.bfloat16, lse_out: Optional[torch.Tensor] = None,
                                 want_lse: bool = True, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Latent attention, expanded form: q [Nq, H, Dn + 64], w_uk [H, Dn, R], w_uv
    [H, Dv, R]; returns (out [Nq, H, Dv], lse [Nq, H])."""
    nb, bs, r = _latent_dims(latent_cache)
    if w_uk.dim() != 3 or w_uv.dim() != 3:
        raise ValueError("w_uk and w_uv must be [num_heads, width, latent_dim]")
    dn, dv = w_uk.shape[1], w_uv.shape[1]
    B, columns = block_tables.shape
    nq, h, out, code, lse_out = _latent_call(q, dn + KF_ROPE_DIM, dv, B, context_lens, q_start, out, out_dtype,
                                             lse_out, want_lse)
    _shape(w_uk, (h, dn, r), "w_uk")
    _shape(w_uv, (h, dv, r), "w_uv")
    dev = q.get_device()
    _call("kf_latent_attention_expanded", dev, stream,
          _on(dev, q, torch.bfloat16, "q"), None if q_start is None else _on(dev, q_start, torch.int32, "q_start"),
          _on(dev, latent_cache, torch.bfloat16, "latent_cache"), _on(dev, w_uk, torch.bfloat16, "w_uk"),
          _on(dev, w_uv, torch.bfloat16, "w_uv"), _on(dev, block_tables, torch.int32, "block_tables"), columns,
          _on(dev, context_lens, torch.int32, "context_lens"), 1 if causal else 0, int(max_context_len),
          int(max_query_len), B, nq, h, r, KF_ROPE_DIM, dn, dv, bs, nb, float(scale),
          _on(dev, workspace, torch.uint8, "workspace"), workspace.numel(), _on(dev, out, out.dtype, "out"), code,
          None if lse_out is None else _on(dev, lse_out, torch.float32, "lse_out"))
    return out, lse_out


def _accumulate(name, q, k_cache, k_scale, block_tables, context_lens, max_context_len, scale, lse, scores_out,
                scores_in, q_start, max_query_len, causal, stream):
    nq, hq, d = q.shape
    nb, bs, hkv, kd = k_cache.shape
    if kd != d:
        _shape(k_cache, (nb, bs, hkv, d), "k_cache")
    B, columns = block_tables.shape
    _shape(context_lens, (B,), "context_lens")
    _shape(lse, (nq, hq), "lse")
    out_shape = scores_out.shape
    if len(out_shape) != 2 or out_shape[0] != B:
        raise ValueError("scores_out must be [batch, stride]")
    if scores_in is not None:
        _shape(scores_in, out_shape, "scores_in")
    if q_start is not None:
        _shape(q_start, (B + 1,), "q_start")
    elif nq != B:
        raise ValueError("q must hold one query token a request without q_start")
    dev = q.get_device()
    if k_scale is None:
        keys = (_on(dev, k_cache, torch.bfloat16, "k_cache"),)
    else:
        _shape(k_scale, (hkv,), "k_scale")
        if k_cache.get_device() != dev:
            raise ValueError("k_cache must be on the call's device, cuda:%d, got %s" % (dev, k_cache.device))
        keys = (_dev8(k_cache, "k_cache"), _on(dev, k_scale, torch.float32, "k_scale"))
    _call(name, dev, stream,
          _on(dev, q, torch.bfloat16, "q"), None if q_start is None else _on(dev, q_start, torch.int32, "q_start"),
          *keys, _on(dev, block_tables, torch.int32, "block_tables"), columns,
          _on(dev, context_lens, torch.int32, "context_lens"), 1 if causal else 0, int(max_context_len),
          int(max_query_len), B, nq, hq, hkv, d, bs, nb, float(scale), _on(dev, lse, torch.float32, "lse"),
          None if scores_in is None else _on(dev, scores_in, torch.float32, "scores_in"),
          _on(dev, scores_out, torch.float32, "scores_out"), out_shape[1])
    return scores_out


def kf_accumulate_attention(q: torch.Tensor, k_cache: torch.Tensor, block_tables: torch.Tensor,
                            context_lens: torch.Tensor, max_context_len: int, scale: float, lse: torch.Tensor,
                            scores_out: torch.Tensor, scores_in: Optional[torch.Tensor] = None,
                            q_start: Optional[torch.Tensor] = None, max_query_len: int = 1, causal: bool = True,
                            stream=None) -> torch.Tensor:
    """scores_out[b, t] = scores_in[b, t] + the attention weight token t receives
    from the queries q [Nq, Hq, D] whose log-sum-exp is lse [Nq, Hq]; scores_out
    [B, stride] may be scores_in (None: zeros). Returns scores_out."""
    return _accumulate("kf_accumulate_attention", q, k_cache, None, block_tables, context_lens, max_context_len,
                       scale, lse, scores_out, scores_in, q_start, max_query_len, causal, stream)


def kf_accumulate_attention_fp8(q, k_cache, k_scale, block_tables, context_lens, max_context_len: int,
                                scale: float, lse, scores_out, scores_in=None, q_start=None, max_query_len: int = 1,
                                causal: bool = True, stream=None) -> torch.Tensor:
    """kf_accumulate_attention over an E4M3 key cache."""
    return _accumulate("kf_accumulate_attention_fp8", q, k_cache, k_scale, block_tables, context_lens,
                       max_context_len, scale, lse, scores_out, scores_in, q_start, max_query_len, causal, stream)


def kf_evict_workspace_size(batch: int, max_context_len: int, keep: int) -> int:
    return int(_lib.kf_evict_workspace_size(batch, max_context_len, keep))


def make_evict_workspace(batch: int, max_context_len: int, keep: int, device=None) -> torch.Tensor:
    """A workspace for kf_evict_tokens (any contents)."""
    n = kf_evict_workspace_size(batch, max_context_len, keep)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def kf_evict_tokens(caches, block_tables: torch.Tensor, context_lens: torch.Tensor, max_context_len: int,
                    scores: torch.Tensor, keep: int, sink: int, recent: int, context_lens_out: torch.Tensor,
                    scores_out: torch.Tensor, workspace: torch.Tensor, positions: Optional[torch.Tensor] = None,
                    seq_lens: Optional[torch.Tensor] = None, positions_out: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Cut every request to its `keep` tokens of most weight, in place. caches: a
    list of one or two paged caches ([num_blocks, block_size, ...], rows of equal bytes: K and
    V, or a latent cache). The *_out tensors may be their inputs."""
    if isinstance(caches, torch.Tensor) or len(caches) not in (1, 2):
        raise ValueError("caches must be one or two tensors")
    first = caches[0]
    shape = first.shape
    if len(shape) < 3 or (len(caches) == 2 and (caches[1].shape != shape or caches[1].dtype != first.dtype)):
        raise ValueError("caches must share one [num_blocks, block_size, ...] shape and type")
    dev = first.get_device()
    cache_a = _on(dev, first, first.dtype, "caches")
    cache_b = _on(dev, caches[1], first.dtype, "caches") if len(caches) == 2 else None
    B, columns = block_tables.shape
    _shape(context_lens, (B,), "context_lens")
    _shape(context_lens_out, (B,), "context_lens_out")
    width = scores.shape
    if len(width) != 2 or width[0] != B:
        raise ValueError("scores must be [batch, stride]")
    _shape(scores_out, width, "scores_out")
    pos = pos_out = seq = None
    if positions is not None:
        _shape(positions, width, "positions")
        pos = _on(dev, positions, torch.int32, "positions")
    if positions_out is not None:
        _shape(positions_out, width, "positions_out")
        pos_out = _on(dev, positions_out, torch.int32, "positions_out")
    if seq_lens is not None:
        _shape(seq_lens, (B,), "seq_lens")
        seq = _on(dev, seq_lens, torch.int32, "seq_lens")
    _call("kf_evict_tokens", dev, stream,
          cache_a, cache_b, first.stride(1) * first.element_size(), _on(dev, block_tables, torch.int32, "block_tables"),
          columns, _on(dev, context_lens, torch.int32, "context_lens"), int(max_context_len), B, shape[1], shape[0],
          _on(dev, scores, torch.float32, "scores"), _on(dev, scores_out, torch.float32, "scores_out"), width[1],
          pos, pos_out, seq, int(keep), int(sink), int(recent),
          _on(dev, context_lens_out, torch.int32, "context_lens_out"), _on(dev, workspace, torch.uint8, "workspace"),
          workspace.numel())


def kf_check_bounded_wait(stream=None) -> None:
    """Launch one bounded wait that nothing completes (sets KF_DEVERR_TIMEOUT)."""
    _check(_lib.kf_check_bounded_wait(_stream(stream)), "kf_check_bounded_wait")


def kf_get_device_error(stream=None) -> int:
    """Synchronise the stream, return and clear the device error word (0 = none)."""
    flags = ctypes.c_uint(0)
    st = _lib.kf_get_device_error(ctypes.byref(flags), _stream(stream))
    if st not in (KF_OK, KF_ERR_DEVICE):
        raise KfError(st, "kf_get_device_error")
    return flags.value
