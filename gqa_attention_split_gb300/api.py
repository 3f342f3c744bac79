"""ctypes binding for libgqa_attn.so — argument marshalling only.

The functions named ``gqa_attn_*`` mirror the C ABI in ``include/gqa_attn.h``
one to one (raw device pointers as ints, sizes, a ``cudaStream_t`` as an int).
``decode`` and ``prefill`` are conveniences over them for torch tensors: they
check dtype/shape/device, allocate outputs, pass ``data_ptr()`` and the current
stream, and raise ``GqaError`` on a non-zero return code. Every step of the
computation runs in the library's CUDA kernels; nothing here computes.

The library must be built first (``python -m gqa_attention_split_gb300.build``
or ``__graft_entry__.build()``); loading fails loudly otherwise.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgqa_attn.so")

GQA_OK = 0
GQA_ERR_INVALID_ARG = -1
GQA_ERR_UNSUPPORTED = -2
GQA_ERR_MISALIGNED = -3
GQA_ERR_CUDA = -4
GQA_ERR_DEVICE_TIMEOUT = -5
GQA_ERR_WORKSPACE = -6
GQA_ERR_DEVICE_BAD_INPUT = -7

# name -> (restype, argtypes); every symbol include/gqa_attn.h declares.
_P, _I, _F, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L = ctypes.c_int64
_SIGNATURES = {
    "gqa_attn_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "gqa_attn_decode_ws": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _S,
                                _P]),
    "gqa_attn_decode_workspace_size": (_S, [_I, _I, _I, _I]),
    "gqa_attn_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "gqa_attn_decode_partial": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I,
                                     _P]),
    "gqa_attn_merge": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "gqa_attn_ring_append": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "gqa_attn_quantize_kv_q8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "gqa_attn_decode_q8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "gqa_attn_decode_ring": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "gqa_attn_prefill": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "gqa_attn_prefill_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P]),
    "gqa_attn_prefill_partial": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                      _F, _P]),
    "gqa_attn_prefill_packed": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _L, _L,
                                     _L, _L, _L, _L, _I, _F, _P]),
    "gqa_attn_decode_tree": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                  _I, _I, _L, _L, _L, _L, _L, _L, _F, _P, _S, _P]),
    "gqa_attn_decode_tree_workspace_size": (_S, [_I, _I, _I, _I]),
    "gqa_attn_cache_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _L, _L,
                                   _L, _L, _P]),
    "gqa_attn_qk_norm_rope": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                   _I, _I, _F, _L, _L, _L, _L, _L, _L, _L, _L, _P]),
    "gqa_attn_paged_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                                   _L, _L, _L, _L, _L, _L, _P]),
    "gqa_attn_paged_attention": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                      _I, _I, _I, _L, _L, _L, _L, _I, _F, _P, _S, _P]),
    "gqa_attn_paged_attention_workspace_size": (_S, [_I, _I, _I, _I]),
    "gqa_attn_verify_drafts": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _L, _L, _P]),
    "gqa_attn_pick_num_splits": (_I, [_I, _I, _I, _I]),
    "gqa_attn_pick_num_splits_q8": (_I, [_I, _I, _I, _I]),
    "gqa_attn_pick_num_splits_q4": (_I, [_I, _I, _I, _I]),
    "gqa_attn_quantize_kv_q4": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "gqa_attn_decode_q4": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "gqa_attn_decode_cluster_size": (_I, [_I, _I, _I, _I]),
    "gqa_attn_split_bounds": (_I, [_I, _I, _I, _P, _P]),
    "gqa_attn_tile_class": (_I, [_I, _I, _I, _I]),
    "gqa_attn_prefill_tile_counts": (_I, [_I, _I, _I, _I, _P, _P, _P]),
    "gqa_attn_prefill_block_m": (_I, []),
    "gqa_attn_prefill_block_n": (_I, []),
    "gqa_attn_prefill_schedule": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _I]),
    "gqa_attn_check": (_I, [_P]),
    "gqa_attn_debug_inject_timeout": (_I, [_I]),
    "gqa_attn_debug_tile_counts": (_I, [_P, _I]),
    "gqa_attn_debug_prefill_order": (_I, [ctypes.c_int64]),
    "gqa_attn_strerror": (ctypes.c_char_p, [_I]),
    "gqa_attn_version": (_I, []),
}

_lib = None
_lock = threading.Lock()


class GqaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (code {code})")


def load(path: str) -> ctypes.CDLL:
    """Loads a build of the library at ``path`` with every signature set.
    ``lib()`` uses it for the product library; tests use it for the debug
    build (``build.build(debug=True)``), which loads beside it."""
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with "
            "`python -m gqa_attention_split_gb300.build` (CUDA 13, sm_103a)")
    L = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


def lib() -> ctypes.CDLL:
    """Loads libgqa_attn.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            _lib = load(LIB_PATH)
    return _lib


def symbols():
    return list(_SIGNATURES)


# ---- one-to-one C ABI mirrors --------------------------------------------


def gqa_attn_decode(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, S_max, scale, num_splits,
                    stream):
    return lib().gqa_attn_decode(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, S_max, scale,
                                 num_splits, stream)


def gqa_attn_decode_ws(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, S_max, scale, num_splits,
                       workspace, workspace_bytes, stream):
    return lib().gqa_attn_decode_ws(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, S_max, scale,
                                    num_splits, workspace, workspace_bytes, stream)


def gqa_attn_decode_noalloc(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, S_max, scale,
                            num_splits, stream):
    return lib().gqa_attn_decode_noalloc(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, S_max,
                                         scale, num_splits, stream)


NOALLOC_SCRATCH_BYTES = 8 << 20  # GQA_NOALLOC_SCRATCH_BYTES


def gqa_attn_decode_workspace_size(B, H_q, d, num_splits):
    return lib().gqa_attn_decode_workspace_size(B, H_q, d, num_splits)


def gqa_attn_prefill(q, k, v, o, lse, B, T_q, S_kv, q_offset, causal, scale, stream):
    return lib().gqa_attn_prefill(q, k, v, o, lse, B, T_q, S_kv, q_offset, causal, scale,
                                  stream)


def gqa_attn_prefill_ex(q, k, v, o, lse, B, H_q, H_kv, d, T_q, S_kv, q_offset, causal, scale,
                        stream):
    return lib().gqa_attn_prefill_ex(q, k, v, o, lse, B, H_q, H_kv, d, T_q, S_kv, q_offset,
                                     causal, scale, stream)


def gqa_attn_prefill_partial(q, k, v, o_part, lse_part, B, H_q, H_kv, d, T_q, S_kv, q_offset,
                             key_offset, causal, scale, stream):
    return lib().gqa_attn_prefill_partial(q, k, v, o_part, lse_part, B, H_q, H_kv, d, T_q, S_kv,
                                          q_offset, key_offset, causal, scale, stream)


def gqa_attn_pick_num_splits(B, H_kv, S_max, num_sms):
    return lib().gqa_attn_pick_num_splits(B, H_kv, S_max, num_sms)


def gqa_attn_pick_num_splits_q8(B, H_kv, S_max, num_sms):
    return lib().gqa_attn_pick_num_splits_q8(B, H_kv, S_max, num_sms)


def gqa_attn_pick_num_splits_q4(B, H_kv, S_max, num_sms):
    return lib().gqa_attn_pick_num_splits_q4(B, H_kv, S_max, num_sms)


def gqa_attn_quantize_kv_q4(k, v, k_codes, v_codes, k_scales, v_scales, B, H_kv, S, d, stream):
    return lib().gqa_attn_quantize_kv_q4(k, v, k_codes, v_codes, k_scales, v_scales, B, H_kv, S,
                                         d, stream)


def gqa_attn_decode_q4(q, k_codes, v_codes, k_scales, v_scales, o, lse, seqlens, B, H_q, H_kv, d,
                       S_max, scale, num_splits, stream):
    return lib().gqa_attn_decode_q4(q, k_codes, v_codes, k_scales, v_scales, o, lse, seqlens, B,
                                    H_q, H_kv, d, S_max, scale, num_splits, stream)


def gqa_attn_decode_cluster_size(B, H_kv, num_splits, num_sms):
    return lib().gqa_attn_decode_cluster_size(B, H_kv, num_splits, num_sms)


def gqa_attn_split_bounds(S_max, num_splits, seqlen):
    """Returns (rc, [(start, end), ...])."""
    starts = (ctypes.c_int32 * max(num_splits, 1))()
    ends = (ctypes.c_int32 * max(num_splits, 1))()
    rc = lib().gqa_attn_split_bounds(S_max, num_splits, seqlen, starts, ends)
    return rc, [(starts[i], ends[i]) for i in range(max(num_splits, 0))] if rc == 0 else []


def gqa_attn_tile_class(qs, qe, ks, ke):
    return lib().gqa_attn_tile_class(qs, qe, ks, ke)


def gqa_attn_prefill_tile_counts(T_q, S_kv, q_offset, causal):
    """Returns (rc, n_past, n_partial, n_future)."""
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    rc = lib().gqa_attn_prefill_tile_counts(T_q, S_kv, q_offset, causal, ctypes.byref(a),
                                            ctypes.byref(b), ctypes.byref(c))
    return rc, a.value, b.value, c.value


def gqa_attn_prefill_block_m():
    return lib().gqa_attn_prefill_block_m()


def gqa_attn_prefill_block_n():
    return lib().gqa_attn_prefill_block_n()


def gqa_attn_prefill_schedule(B, H_q, H_kv, d, T_q, S_kv, q_offset, causal, num_ctas,
                              item_cap=12288):
    """Returns (rc, per-CTA item lists); rc = 0 (closed-form order) gives []."""
    off = (ctypes.c_int32 * (num_ctas + 1))()
    items = (ctypes.c_int32 * max(1, item_cap))()
    rc = lib().gqa_attn_prefill_schedule(B, H_q, H_kv, d, T_q, S_kv, q_offset, causal, num_ctas,
                                         off, items, item_cap)
    if rc <= 0:
        return rc, []
    return rc, [list(items[off[c]:off[c + 1]]) for c in range(num_ctas)]


def gqa_attn_check(stream=None):
    return lib().gqa_attn_check(stream)


def gqa_attn_debug_inject_timeout(launches):
    return lib().gqa_attn_debug_inject_timeout(launches)


def gqa_attn_debug_prefill_order(budget_bytes):
    return lib().gqa_attn_debug_prefill_order(budget_bytes)


def gqa_attn_debug_tile_counts(clear=False, L=None):
    """Returns (rc, [all_past, partial, all_future]) from ``L`` (default: the
    product library, whose non-debug build returns GQA_ERR_UNSUPPORTED)."""
    c = (ctypes.c_int64 * 3)()
    rc = (L or lib()).gqa_attn_debug_tile_counts(c, 1 if clear else 0)
    return rc, [c[0], c[1], c[2]]


def strerror(code: int) -> str:
    return lib().gqa_attn_strerror(code).decode()


def gqa_attn_version():
    return lib().gqa_attn_version()


# ---- torch conveniences -----------------------------------------------------


def _stream_ptr(stream=None):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_cuda_bf16(name, t, ndim):
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor, got {tuple(t.shape)}")


def decode(q, k, v, seqlens=None, *, num_splits: int = 0, scale: float | None = None,
           out=None, lse=None, stream=None, workspace=None):
    """Split-KV decode. q [B,H_q,d], k/v [B,H_kv,S_max,d] bf16 CUDA; seqlens int32 [B] or None.

    Returns (o [B,H_q,d] bf16, lse [B,H_q] fp32). With ``workspace`` (a uint8
    CUDA tensor) the call goes through gqa_attn_decode_ws.
    """
    import torch

    _check_cuda_bf16("q", q, 3)
    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    B, H_q, d = q.shape
    H_kv, S_max = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k, v must be [B, H_kv, S_max, d] matching q")
    if seqlens is not None and (seqlens.dtype != torch.int32 or not seqlens.is_cuda
                                or seqlens.numel() != B):
        raise TypeError("seqlens must be an int32 CUDA tensor of B elements")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    st = _stream_ptr(stream)
    if workspace is None:
        rc = gqa_attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(seqlens),
                             B, H_q, H_kv, d, S_max, sc, num_splits, st)
    else:
        rc = gqa_attn_decode_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                _ptr(seqlens), B, H_q, H_kv, d, S_max, sc, num_splits,
                                _ptr(workspace), workspace.numel(), st)
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_decode")
    return out, lse


def gqa_attn_decode_partial(q, k, v, o_part, lse_part, seqlens, B, H_q, H_kv, d, S_max, scale,
                            num_splits, stream):
    return lib().gqa_attn_decode_partial(q, k, v, o_part, lse_part, seqlens, B, H_q, H_kv, d,
                                         S_max, scale, num_splits, stream)


def gqa_attn_merge(o_parts, lse_parts, o, lse, R, rows, d, stream):
    return lib().gqa_attn_merge(o_parts, lse_parts, o, lse, R, rows, d, stream)


def decode_partial(q, k, v, seqlens=None, *, num_splits: int = 0, scale: float | None = None,
                   out=None, lse=None, stream=None):
    """Decode over one key slice with fp32 output for ``merge``: q [B,H_q,d],
    k/v [B,H_kv,S_slice,d] bf16 CUDA. Returns (o fp32 [B,H_q,d], lse [B,H_q])."""
    import torch

    _check_cuda_bf16("q", q, 3)
    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    B, H_q, d = q.shape
    H_kv, S_max = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k, v must be [B, H_kv, S, d] matching q")
    if seqlens is not None and (seqlens.dtype != torch.int32 or not seqlens.is_cuda
                                or seqlens.numel() != B):
        raise TypeError("seqlens must be an int32 CUDA tensor of B elements")
    if out is None:
        out = torch.empty((B, H_q, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = gqa_attn_decode_partial(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(seqlens),
                                 B, H_q, H_kv, d, S_max, sc, num_splits, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_decode_partial")
    return out, lse


def merge(o_parts, lse_parts, *, out=None, lse=None, stream=None):
    """Log-sum-exp merge of R partials: o_parts fp32 [R, ..., d], lse_parts
    fp32 [R, ...] (CUDA, contiguous). Returns (o bf16 [..., d], lse [...])."""
    import torch

    if (o_parts.dtype != torch.float32 or lse_parts.dtype != torch.float32 or not o_parts.is_cuda
            or not o_parts.is_contiguous() or not lse_parts.is_contiguous()
            or tuple(o_parts.shape[:-1]) != tuple(lse_parts.shape)):
        raise ValueError("o_parts [R, ..., d] and lse_parts [R, ...] must be contiguous fp32 CUDA")
    R, d = o_parts.shape[0], o_parts.shape[-1]
    rows = lse_parts[0].numel()
    if out is None:
        out = torch.empty(tuple(o_parts.shape[1:]), dtype=torch.bfloat16, device=o_parts.device)
    if lse is None:
        lse = torch.empty(tuple(lse_parts.shape[1:]), dtype=torch.float32, device=o_parts.device)
    rc = gqa_attn_merge(_ptr(o_parts), _ptr(lse_parts), _ptr(out), _ptr(lse), R, rows, d,
                        _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_merge")
    return out, lse


def gqa_attn_ring_append(k_cache, v_cache, k_new, v_new, positions, B, H_kv, d, capacity, n_sink,
                         stream):
    return lib().gqa_attn_ring_append(k_cache, v_cache, k_new, v_new, positions, B, H_kv, d,
                                      capacity, n_sink, stream)


def gqa_attn_decode_ring(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, capacity, n_sink, scale,
                         num_splits, stream):
    return lib().gqa_attn_decode_ring(q, k, v, o, lse, seqlens, B, H_q, H_kv, d, capacity,
                                      n_sink, scale, num_splits, stream)


def gqa_attn_quantize_kv_q8(k, v, k_codes, v_codes, k_scales, v_scales, B, H_kv, S, d, stream):
    return lib().gqa_attn_quantize_kv_q8(k, v, k_codes, v_codes, k_scales, v_scales, B, H_kv, S,
                                         d, stream)


def gqa_attn_decode_q8(q, k_codes, v_codes, k_scales, v_scales, o, lse, seqlens, B, H_q, H_kv, d,
                       S_max, scale, num_splits, stream):
    return lib().gqa_attn_decode_q8(q, k_codes, v_codes, k_scales, v_scales, o, lse, seqlens, B,
                                    H_q, H_kv, d, S_max, scale, num_splits, stream)


def quantize_kv_q8(k, v, *, stream=None):
    """INT8 cache from a bf16 cache k, v [B,H_kv,S,d] (CUDA): returns
    (k_codes [B,H_kv,S,d], v_codes [B,H_kv,d,S] as uint8 bytes code + 128,
    k_scales, v_scales [B,H_kv,S] fp32)."""
    import torch

    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    B, H_kv, S, d = k.shape
    kc = torch.empty((B, H_kv, S, d), dtype=torch.uint8, device=k.device)
    vc = torch.empty((B, H_kv, d, S), dtype=torch.uint8, device=k.device)
    ks = torch.empty((B, H_kv, S), dtype=torch.float32, device=k.device)
    vs = torch.empty_like(ks)
    rc = gqa_attn_quantize_kv_q8(_ptr(k), _ptr(v), _ptr(kc), _ptr(vc), _ptr(ks), _ptr(vs), B, H_kv,
                                 S, d, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_quantize_kv_q8")
    return kc, vc, ks, vs


def decode_q8(q, k_codes, v_codes, k_scales, v_scales, seqlens=None, *, num_splits: int = 0,
              scale: float | None = None, out=None, lse=None, stream=None):
    """Split-KV decode over an INT8 cache (layouts as ``quantize_kv_q8``).
    Returns (o [B,H_q,d] bf16, lse [B,H_q] fp32)."""
    import torch

    _check_cuda_bf16("q", q, 3)
    B, H_q, d = q.shape
    H_kv, S_max = k_codes.shape[1], k_codes.shape[2]
    if (k_codes.dtype != torch.uint8 or v_codes.dtype != torch.uint8
            or k_codes.shape != (B, H_kv, S_max, d) or v_codes.shape != (B, H_kv, d, S_max)):
        raise ValueError("k_codes [B,H_kv,S,d] and v_codes [B,H_kv,d,S] must be uint8")
    for nm, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t.dtype != torch.float32 or t.shape != (B, H_kv, S_max) or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous fp32 [B, H_kv, S] tensor")
    if seqlens is not None and (seqlens.dtype != torch.int32 or not seqlens.is_cuda
                                or seqlens.numel() != B):
        raise TypeError("seqlens must be an int32 CUDA tensor of B elements")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = gqa_attn_decode_q8(_ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scales),
                            _ptr(v_scales), _ptr(out), _ptr(lse), _ptr(seqlens), B, H_q, H_kv, d,
                            S_max, sc, num_splits, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_decode_q8")
    return out, lse


def quantize_kv_q4(k, v, *, stream=None):
    """INT4 cache from a bf16 cache k, v [B,H_kv,S,d] (CUDA): returns
    (k_codes [B,H_kv,S,d/2], v_codes [B,H_kv,d,S/2] as uint8, two nibbles
    code + 8 per byte, k_scales, v_scales [B,H_kv,S] fp32)."""
    import torch

    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    B, H_kv, S, d = k.shape
    kc = torch.empty((B, H_kv, S, d // 2), dtype=torch.uint8, device=k.device)
    vc = torch.empty((B, H_kv, d, S // 2), dtype=torch.uint8, device=k.device)
    ks = torch.empty((B, H_kv, S), dtype=torch.float32, device=k.device)
    vs = torch.empty_like(ks)
    rc = gqa_attn_quantize_kv_q4(_ptr(k), _ptr(v), _ptr(kc), _ptr(vc), _ptr(ks), _ptr(vs), B, H_kv,
                                 S, d, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_quantize_kv_q4")
    return kc, vc, ks, vs


def decode_q4(q, k_codes, v_codes, k_scales, v_scales, seqlens=None, *, num_splits: int = 0,
              scale: float | None = None, out=None, lse=None, stream=None):
    """Split-KV decode over an INT4 cache (layouts as ``quantize_kv_q4``).
    Returns (o [B,H_q,d] bf16, lse [B,H_q] fp32)."""
    import torch

    _check_cuda_bf16("q", q, 3)
    B, H_q, d = q.shape
    H_kv, S_max = k_codes.shape[1], k_codes.shape[2]
    if (k_codes.dtype != torch.uint8 or v_codes.dtype != torch.uint8
            or k_codes.shape != (B, H_kv, S_max, d // 2)
            or v_codes.shape != (B, H_kv, d, S_max // 2)):
        raise ValueError("k_codes [B,H_kv,S,d/2] and v_codes [B,H_kv,d,S/2] must be uint8")
    for nm, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t.dtype != torch.float32 or t.shape != (B, H_kv, S_max) or not t.is_contiguous():
            raise ValueError(f"{nm} must be a contiguous fp32 [B, H_kv, S] tensor")
    if seqlens is not None and (seqlens.dtype != torch.int32 or not seqlens.is_cuda
                                or seqlens.numel() != B):
        raise TypeError("seqlens must be an int32 CUDA tensor of B elements")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = gqa_attn_decode_q4(_ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scales),
                            _ptr(v_scales), _ptr(out), _ptr(lse), _ptr(seqlens), B, H_q, H_kv, d,
                            S_max, sc, num_splits, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_decode_q4")
    return out, lse


def ring_append(k_cache, v_cache, k_new, v_new, positions, *, n_sink: int, stream=None):
    """Writes each row's newest token into its ring slot. k_cache/v_cache
    [B,H_kv,capacity,d] bf16 CUDA; k_new/v_new [B,H_kv,d]; positions int32 [B]
    (the new token's index in its row)."""
    import torch

    _check_cuda_bf16("k_cache", k_cache, 4)
    _check_cuda_bf16("v_cache", v_cache, 4)
    _check_cuda_bf16("k_new", k_new, 3)
    _check_cuda_bf16("v_new", v_new, 3)
    B, H_kv, capacity, d = k_cache.shape
    if v_cache.shape != k_cache.shape or k_new.shape != (B, H_kv, d) or v_new.shape != k_new.shape:
        raise ValueError("k_new, v_new must be [B, H_kv, d] matching the caches")
    if positions.dtype != torch.int32 or not positions.is_cuda or positions.numel() != B:
        raise TypeError("positions must be an int32 CUDA tensor of B elements")
    rc = gqa_attn_ring_append(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                              _ptr(positions), B, H_kv, d, capacity, n_sink, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_ring_append")


def decode_ring(q, k, v, seqlens, *, n_sink: int, num_splits: int = 0,
                scale: float | None = None, out=None, lse=None, stream=None):
    """Decode over a ring-buffer cache with attention sinks: k/v
    [B,H_kv,capacity,d]; seqlens int32 [B] counts every token each row has
    produced (it may exceed capacity). Returns (o, lse) as ``decode``."""
    import torch

    _check_cuda_bf16("q", q, 3)
    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    B, H_q, d = q.shape
    H_kv, capacity = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k, v must be [B, H_kv, capacity, d] matching q")
    if seqlens.dtype != torch.int32 or not seqlens.is_cuda or seqlens.numel() != B:
        raise TypeError("seqlens must be an int32 CUDA tensor of B elements")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = gqa_attn_decode_ring(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(seqlens),
                              B, H_q, H_kv, d, capacity, n_sink, sc, num_splits,
                              _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_decode_ring")
    return out, lse


def prefill(q, k, v, *, q_offset: int = 0, causal: bool = True, scale: float | None = None,
            out=None, lse=None, stream=None):
    """Causal (or full) prefill. q [B,H_q,T_q,d], k/v [B,H_kv,S_kv,d] bf16 CUDA.

    Returns (o [B,H_q,T_q,d] bf16, lse [B,H_q,T_q] fp32).
    """
    import torch

    _check_cuda_bf16("q", q, 4)
    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    B, H_q, T_q, d = q.shape
    H_kv, S_kv = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k, v must be [B, H_kv, S_kv, d] matching q")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H_q, T_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = gqa_attn_prefill_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, d,
                             T_q, S_kv, q_offset, 1 if causal else 0, sc, _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_prefill")
    return out, lse


def prefill_partial(q, k, v, *, q_offset: int = 0, key_offset: int = 0, causal: bool = True,
                    scale: float | None = None, out=None, lse=None, stream=None):
    """Prefill against one slice of the keys (global positions key_offset + j),
    O in fp32 for ``merge``. q [B,H_q,T_q,d], k/v [B,H_kv,S_slice,d] bf16 CUDA.
    Returns (o fp32 [B,H_q,T_q,d], lse [B,H_q,T_q])."""
    import torch

    _check_cuda_bf16("q", q, 4)
    _check_cuda_bf16("k", k, 4)
    _check_cuda_bf16("v", v, 4)
    B, H_q, T_q, d = q.shape
    H_kv, S_kv = k.shape[1], k.shape[2]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k, v must be [B, H_kv, S_slice, d] matching q")
    if out is None:
        out = torch.empty((B, H_q, T_q, d), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H_q, T_q), dtype=torch.float32, device=q.device)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = gqa_attn_prefill_partial(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv,
                                  d, T_q, S_kv, q_offset, key_offset, 1 if causal else 0, sc,
                                  _stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_prefill_partial")
    return out, lse


# ---- ragged batches ---------------------------------------------------------


def gqa_attn_prefill_packed(q, k, v, o, lse, cu_q, cu_k, B, H_q, H_kv, d, total_q, total_k,
                            q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t,
                            v_stride_h, causal, scale, stream):
    return lib().gqa_attn_prefill_packed(q, k, v, o, lse, cu_q, cu_k, B, H_q, H_kv, d, total_q,
                                         total_k, q_stride_t, q_stride_h, k_stride_t, k_stride_h,
                                         v_stride_t, v_stride_h, causal, scale, stream)


def gqa_attn_decode_tree(q, k_new, v_new, k_cache, v_cache, o, lse, cu_seqlens, context_lens,
                         tree_mask, mask_words, B, H_q, H_kv, d, total, max_tokens, S_max,
                         q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t, v_stride_h,
                         scale, workspace, workspace_bytes, stream):
    return lib().gqa_attn_decode_tree(q, k_new, v_new, k_cache, v_cache, o, lse, cu_seqlens,
                                      context_lens, tree_mask, mask_words, B, H_q, H_kv, d, total,
                                      max_tokens, S_max, q_stride_t, q_stride_h, k_stride_t,
                                      k_stride_h, v_stride_t, v_stride_h, scale, workspace,
                                      workspace_bytes, stream)


def gqa_attn_decode_tree_workspace_size(H_q, H_kv, d, max_tokens):
    return lib().gqa_attn_decode_tree_workspace_size(H_q, H_kv, d, max_tokens)


def gqa_attn_cache_append(k_cache, v_cache, k_new, v_new, cu_seqlens, starts, index, B, H_kv, d,
                          S_max, total, total_new, k_stride_t, k_stride_h, v_stride_t, v_stride_h,
                          stream):
    return lib().gqa_attn_cache_append(k_cache, v_cache, k_new, v_new, cu_seqlens, starts, index,
                                       B, H_kv, d, S_max, total, total_new, k_stride_t, k_stride_h,
                                       v_stride_t, v_stride_h, stream)


def gqa_attn_qk_norm_rope(q, k, q_out, k_out, q_weight, k_weight, weights_fp32, positions,
                          inv_freq, sections, axes, tokens, H_q, H_kv, d, pairs, interleaved, norm,
                          eps, q_stride_t, q_stride_h, k_stride_t, k_stride_h, qo_stride_t,
                          qo_stride_h, ko_stride_t, ko_stride_h, stream):
    """``sections``: a list of host ints, or None with one axis."""
    sec = None if sections is None else (ctypes.c_int32 * len(sections))(*sections)
    return lib().gqa_attn_qk_norm_rope(q, k, q_out, k_out, q_weight, k_weight, weights_fp32,
                                       positions, inv_freq, sec, axes, tokens, H_q, H_kv, d, pairs,
                                       interleaved, norm, eps, q_stride_t, q_stride_h, k_stride_t,
                                       k_stride_h, qo_stride_t, qo_stride_h, ko_stride_t,
                                       ko_stride_h, stream)


def gqa_attn_paged_append(k_pages, v_pages, k_new, v_new, cu_seqlens, starts, index, block_table,
                          B, H_kv, d, total, total_new, num_pages, page_size, table_width,
                          k_stride_t, k_stride_h, v_stride_t, v_stride_h, k_page_stride,
                          v_page_stride, stream):
    return lib().gqa_attn_paged_append(k_pages, v_pages, k_new, v_new, cu_seqlens, starts, index,
                                       block_table, B, H_kv, d, total, total_new, num_pages,
                                       page_size, table_width, k_stride_t, k_stride_h, v_stride_t,
                                       v_stride_h, k_page_stride, v_page_stride, stream)


def gqa_attn_paged_attention(q, k_pages, v_pages, o, lse, cu_seqlens, kv_lens, block_table, B, H_q,
                             H_kv, d, total, max_tokens, max_keys, num_pages, page_size,
                             table_width, q_stride_t, q_stride_h, k_page_stride, v_page_stride,
                             causal, scale, workspace, workspace_bytes, stream):
    return lib().gqa_attn_paged_attention(q, k_pages, v_pages, o, lse, cu_seqlens, kv_lens,
                                          block_table, B, H_q, H_kv, d, total, max_tokens,
                                          max_keys, num_pages, page_size, table_width, q_stride_t,
                                          q_stride_h, k_page_stride, v_page_stride, causal, scale,
                                          workspace, workspace_bytes, stream)


def gqa_attn_paged_attention_workspace_size(H_q, H_kv, d, max_tokens):
    return lib().gqa_attn_paged_attention_workspace_size(H_q, H_kv, d, max_tokens)


def gqa_attn_verify_drafts(target_probs, draft_probs, draft_tokens, u_accept, u_sample, cu_seqlens,
                           accepted, next_tokens, B, total, V, target_stride, draft_stride,
                           stream):
    return lib().gqa_attn_verify_drafts(target_probs, draft_probs, draft_tokens, u_accept,
                                        u_sample, cu_seqlens, accepted, next_tokens, B, total, V,
                                        target_stride, draft_stride, stream)


# The checks below run on every call of a serving step whose kernels take a few microseconds, so
# they ask each tensor as little as they can (get_device is -1 for a CPU tensor).


def _packed(torch, name, t, heads, d, device):
    """Checks a packed [tokens, heads, d] bf16 tensor (heads, d or device None: any); returns its
    token and head strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or (
            d is not None and shape[2] != d):
        want = f"[tokens, {'heads' if heads is None else heads}, {'d' if d is None else d}]"
        raise ValueError(f"{name} must be {want}, got {tuple(shape)}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # the stride of a dimension of size 1 says nothing: any valid one will do
    return (st if shape[0] > 1 else 8), (sh if shape[1] > 1 else 8)


def _ints(torch, name, t, n, device):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return t.data_ptr()


def _cache(torch, k_cache, v_cache, H_kv, d, device):
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.bfloat16:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"{name} must be contiguous and on cuda:{device}")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or shape[1] != H_kv or shape[3] != d:
        raise ValueError(f"k_cache, v_cache must be [B, {H_kv}, S_max, {d}]")
    return shape[0], shape[2]


def _outputs(torch, q, out, lse, stream=None):
    if stream is not None and (out is None or lse is None):
        # from the launch stream's pool: what the current stream still reads is not overwritten
        with torch.cuda.stream(stream):
            return _outputs(
                torch, q,
                torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if out is None else out,
                torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
                if lse is None else lse)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    elif (out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous()
          or out.get_device() != q.get_device()):
        raise ValueError("out must be a contiguous bfloat16 tensor shaped like q on its device")
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    elif (lse.dtype is not torch.float32 or lse.shape != q.shape[:2] or not lse.is_contiguous()
          or lse.get_device() != q.get_device()):
        raise ValueError("lse must be a contiguous float32 [tokens, H_q] tensor on q's device")
    return out, lse


def _on_device(torch, device, call):
    """Runs call() with ``device`` current."""
    if torch._C._cuda_getDevice() == device:
        return call()
    with torch.cuda.device(device):
        return call()


def _raw_stream(torch, device, stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


def _in_use(torch, device, stream, *tensors):
    """Tells the allocator that ``tensors`` are used on ``stream`` and on the current stream, so that
    memory freed by one of them is not handed out while the other still works on it."""
    current = torch.cuda.current_stream(device)
    if stream == current:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
            t.record_stream(current)


def prefill_packed(q, k, v, cu_seqlens, cu_seqlens_k=None, *, causal: bool = True,
                   scale: float | None = None, out=None, lse=None, stream=None):
    """Attention over packed sequences of different lengths. q [total_q,H_q,d], k/v
    [total_k,H_kv,d] bf16 CUDA (any token and head strides that are positive multiples of 8, so
    slices of a fused projection are taken as they are); cu_seqlens, cu_seqlens_k int32 [B+1] prefix
    sums of the query and key counts (cu_seqlens_k None: the same). The queries of a sequence are its
    last tokens: causal query t sees keys j <= n_k - n_q + t. A block of queries runs all its keys on
    one SM: few queries on many keys are served faster by decode or decode_tree.

    Returns (o [total_q,H_q,d] bf16, lse [total_q,H_q] fp32). Rows behind the last sequence are
    not written. The call runs on ``stream`` (default: the current stream of q's device); waiting
    for what the current stream still writes to the inputs, and for the results, is the caller's,
    but memory freed on either stream is not reused before the other is done with it.
    """
    import torch

    qs, qh = _packed(torch, "q", q, None, None, None)
    total_q, H_q, d = q.shape
    dev = q.get_device()
    ks, kh = _packed(torch, "k", k, None, d, dev)
    total_k, H_kv, _ = k.shape
    vs, vh = _packed(torch, "v", v, H_kv, d, dev)
    if v.shape[0] != total_k:
        raise ValueError("k and v must have the same shape")
    B = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else 0
    if B < 0:
        raise ValueError("cu_seqlens must have B + 1 elements")
    cu_q = _ints(torch, "cu_seqlens", cu_seqlens, B + 1, dev)
    cu_k = None
    if cu_seqlens_k is not None:
        cu_k = _ints(torch, "cu_seqlens_k", cu_seqlens_k, B + 1, dev)
    elif total_k != total_q:
        raise ValueError("k and v must have q's tokens when cu_seqlens_k is not given")
    out, lse = _outputs(torch, q, out, lse, stream)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_prefill_packed(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), cu_q, cu_k, B,
        H_q, H_kv, d, total_q, total_k, qs, qh, ks, kh, vs, vh, 1 if causal else 0, sc,
        _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_prefill_packed")
    if stream is not None:
        _in_use(torch, dev, stream, q, k, v, out, lse, cu_seqlens, cu_seqlens_k)
    return out, lse


def decode_tree(q, k_new, v_new, k_cache, v_cache, context_lens, *, cu_seqlens=None,
                max_tokens: int | None = None, tree_mask=None, scale: float | None = None,
                out=None, lse=None, stream=None, workspace=None):
    """Attention of drafted tokens over the cache: row b has context_lens[b] (int32 [B]) tokens in
    k_cache/v_cache [B,H_kv,S_max,d] and its drafted tokens packed in q [total,H_q,d],
    k_new/v_new [total,H_kv,d] (prefix sums cu_seqlens int32 [B+1]; None: total / B per row).
    A drafted token sees its row's context and the drafted tokens whose bits are set in its row of
    tree_mask (int32 [total, words], bit j for the row's token j), or with tree_mask None those
    up to itself. max_tokens (at most 128) bounds a row's drafted tokens; it is needed with
    cu_seqlens, whose values stay on the device.

    Returns (o [total,H_q,d] bf16, lse [total,H_q] fp32). ``workspace``: a uint8 CUDA tensor of
    gqa_attn_decode_tree_workspace_size bytes that no overlapping call uses; by default one is
    allocated for the call.
    """
    import torch

    qs, qh = _packed(torch, "q", q, None, None, None)
    total, H_q, d = q.shape
    dev = q.get_device()
    ks, kh = _packed(torch, "k_new", k_new, None, d, dev)
    H_kv = k_new.shape[1]
    vs, vh = _packed(torch, "v_new", v_new, H_kv, d, dev)
    if v_new.shape[0] != total or k_new.shape[0] != total:
        raise ValueError("k_new, v_new must be [total, H_kv, d] with q's tokens")
    B, S_max = _cache(torch, k_cache, v_cache, H_kv, d, dev)
    ctx = _ints(torch, "context_lens", context_lens, B, dev)
    cu = None
    if cu_seqlens is not None:
        cu = _ints(torch, "cu_seqlens", cu_seqlens, B + 1, dev)
        if max_tokens is None:
            raise ValueError("max_tokens is needed with cu_seqlens")
    else:
        if B == 0 or total % B:
            raise ValueError("without cu_seqlens every row has total / B drafted tokens")
        max_tokens = max(1, total // B) if max_tokens is None else max_tokens
    words, mask = 0, None
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != total:
            raise ValueError("tree_mask must be a contiguous int32 [total, words] tensor")
        words = tree_mask.shape[1]
        mask = _ints(torch, "tree_mask", tree_mask, total * words, dev)
    out, lse = _outputs(torch, q, out, lse, stream)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    given = workspace
    if workspace is None:
        # from the launch stream's pool: its memory is reused only behind this call
        n = lib().gqa_attn_decode_tree_workspace_size(H_q, H_kv, d, max_tokens)
        if stream is None:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{dev}")
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_decode_tree(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        out.data_ptr(), lse.data_ptr(), cu, ctx, mask, words, B, H_q, H_kv, d, total, max_tokens,
        S_max, qs, qh, ks, kh, vs, vh, sc, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_decode_tree")
    if stream is not None:
        _in_use(torch, dev, stream, q, k_new, v_new, k_cache, v_cache, out, lse, context_lens,
                cu_seqlens, tree_mask, given)
    return out, lse


def cache_append(k_cache, v_cache, k_new, v_new, starts, *, cu_seqlens=None, index=None,
                 stream=None):
    """Writes packed tokens into the cache k_cache/v_cache [B,H_kv,S_max,d]: entry i of row b (the
    packed entry cu_seqlens[b] + i; cu_seqlens None: the same number for every row) goes to slot
    starts[b] + i (int32 [B]). Entry e is token e of k_new/v_new [tokens,H_kv,d], or token
    index[e] (int32) when index is given, such as the accepted path of a drafted tree."""
    import torch

    ks, kh = _packed(torch, "k_new", k_new, None, None, None)
    total_new, H_kv, d = k_new.shape
    dev = k_new.get_device()
    vs, vh = _packed(torch, "v_new", v_new, H_kv, d, dev)
    if v_new.shape[0] != total_new:
        raise ValueError("k_new and v_new must have the same shape")
    B, S_max = _cache(torch, k_cache, v_cache, H_kv, d, dev)
    first = _ints(torch, "starts", starts, B, dev)
    total, idx, cu = total_new, None, None
    if index is not None:
        total = index.numel() if isinstance(index, torch.Tensor) else 0
        idx = _ints(torch, "index", index, total, dev)
    if cu_seqlens is not None:
        cu = _ints(torch, "cu_seqlens", cu_seqlens, B + 1, dev)
    elif B == 0 or total % B:
        raise ValueError("without cu_seqlens every row has the same number of entries")
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_cache_append(
        k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), cu, first, idx,
        B, H_kv, d, S_max, total, total_new, ks, kh, vs, vh, _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_cache_append")
    if stream is not None:
        _in_use(torch, dev, stream, k_cache, v_cache, k_new, v_new, starts, cu_seqlens, index)


def _empty(torch, t, shape, dtype, stream):
    """New memory beside t, from the launch stream's pool: what the current stream still reads is
    not overwritten."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=t.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=t.device)


def _counts(torch, name, t, given, n):
    if (given.dtype is not torch.int32 or given.shape != (n,) or not given.is_contiguous()
            or given.get_device() != t.get_device()):
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on {t.device}")
    return given


def _weight(torch, name, t, d, device):
    wide = isinstance(t, torch.Tensor) and t.dtype is torch.float32
    if not wide and not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16):
        raise TypeError(f"{name} must be a bfloat16 or float32 CUDA tensor")
    if t.get_device() != device or t.dim() != 1 or t.numel() != d or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{d}] tensor on cuda:{device}")
    return wide


@functools.lru_cache(maxsize=256)
def _paged_workspace(H_q, H_kv, d, max_tokens):
    return lib().gqa_attn_paged_attention_workspace_size(H_q, H_kv, d, max_tokens)


def _floats(torch, name, t, n, device):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, got {t.numel()}")
    return t.data_ptr()


def _pages(torch, k_pages, v_pages, block_table, H_kv, d, device):
    """Checks pages [num_pages, H_kv, page_size, d] and the block table [B, width]; returns
    (B, num_pages, page_size, width, K page stride, V page stride, H_kv, table pointer)."""
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError(f"k_pages, v_pages must be [num_pages, {H_kv or 'H_kv'}, page_size, {d}]")
    n, heads, size, width = shape
    if width != d or (H_kv is not None and heads != H_kv):
        raise ValueError(f"k_pages, v_pages must be [num_pages, {H_kv or 'H_kv'}, page_size, {d}]")
    kp, kh, ks, kd = k_pages.stride()
    vp, vh, vs, vd = v_pages.stride()
    if (kd != 1 or vd != 1 or (size > 1 and (ks != d or vs != d))
            or (heads > 1 and (kh != size * d or vh != size * d))):
        raise ValueError("every page of k_pages and v_pages must be contiguous")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise TypeError("block_table must be a contiguous int32 [B, width] CUDA tensor")
    B, width = block_table.shape
    return B, n, size, width, kp, vp, heads, _ints(torch, "block_table", block_table, B * width,
                                                   device)


def qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None,
                 eps: float | None = 1e-6, sections=None, interleaved: bool = False, q_out=None,
                 k_out=None, stream=None):
    """Norm and rotation of queries q [tokens,H_q,d] and keys k [tokens,H_kv,d] (bf16, strides as
    prefill_packed; k None: queries alone) in one pass. Every head is divided by its root mean
    square sqrt(mean + eps) and multiplied by q_weight / k_weight ([d] bf16 or float32, None: 1);
    eps None leaves the norm and the weights out. Pair i of the inv_freq.numel() pairs of channels,
    (i, i + pairs) or with interleaved (2i, 2i + 1), is then turned by positions * inv_freq[i]
    (float32 [pairs], a multiple of 8 up to d / 2); the channels behind them are left as they are.

    positions: int32 [tokens], or [axes,tokens] with sections, a tuple of the numbers of pairs that
    each axis turns (time, height and width of images and video; at most 4). q_out, k_out may be q
    and k themselves. Returns (q_out, k_out), new contiguous tensors by default. ``stream`` as
    prefill_packed."""
    import torch

    qs, qh = _packed(torch, "q", q, None, None, None)
    n, H_q, d = q_shape = q.shape
    dev = q.get_device()
    ks = kh = kos = koh = 8
    H_kv = 0
    if k is not None:
        ks, kh = _packed(torch, "k", k, None, d, dev)
        n_k, H_kv, _ = k_shape = k.shape
        if n_k != n:
            raise ValueError("q and k must have the same tokens")
        if H_kv == 0:
            raise ValueError("k has no heads")
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    pairs = inv_freq.numel() if isinstance(inv_freq, torch.Tensor) else 0
    freq = _floats(torch, "inv_freq", inv_freq, pairs, dev)
    if sections is None:
        axes, sec = 1, None
    else:
        axes = len(sections)
        sec = (ctypes.c_int32 * axes)(*sections)
    pos = _ints(torch, "positions", positions, axes * n, dev)
    if positions.dim() != (1 if sections is None else 2) or positions.shape[-1] != n:
        raise ValueError(f"positions must be {'[tokens]' if sections is None else '[axes, tokens]'}"
                         f", got {tuple(positions.shape)}")
    qw = kw = wide = None
    if q_weight is not None:
        wide = _weight(torch, "q_weight", q_weight, d, dev)
        qw = q_weight.data_ptr()
    if k_weight is not None:
        wide_k = _weight(torch, "k_weight", k_weight, d, dev)
        if wide is not None and wide != wide_k:
            raise TypeError("q_weight and k_weight must have one type")
        wide, kw = wide_k, k_weight.data_ptr()
    if eps is None and wide is not None:
        raise ValueError("weights need the norm (eps)")
    if q_out is None:
        q_out = _empty(torch, q, q_shape, torch.bfloat16, stream)
        qos, qoh = H_q * d, d
    else:
        if q_out.shape != q_shape:
            raise ValueError("q_out must be shaped like q")
        qos, qoh = _packed(torch, "q_out", q_out, H_q, d, dev)
    k_ptr = ko_ptr = None
    if k is not None:
        if k_out is None:
            k_out = _empty(torch, k, k_shape, torch.bfloat16, stream)
            kos, koh = H_kv * d, d
        else:
            if k_out.shape != k_shape:
                raise ValueError("k_out must be shaped like k")
            kos, koh = _packed(torch, "k_out", k_out, H_kv, d, dev)
        k_ptr, ko_ptr = k.data_ptr(), k_out.data_ptr()
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_qk_norm_rope(
        q.data_ptr(), k_ptr, q_out.data_ptr(), ko_ptr, qw, kw, 1 if wide else 0, pos, freq, sec,
        axes, n, H_q, H_kv, d, pairs, 1 if interleaved else 0, 0 if eps is None else 1,
        0.0 if eps is None else eps, qs, qh, ks, kh, qos, qoh, kos, koh,
        _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_qk_norm_rope")
    if stream is not None:
        _in_use(torch, dev, stream, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    return q_out, k_out


def paged_append(k_pages, v_pages, k_new, v_new, block_table, starts, *, cu_seqlens=None,
                 index=None, stream=None):
    """cache_append over pages k_pages/v_pages [num_pages,H_kv,page_size,d] (each page contiguous;
    page_size 16, 32, 64 or a multiple of 128): slot s of row b lies in page
    block_table[b, s // page_size] (int32 [B,width])."""
    import torch

    ks, kh = _packed(torch, "k_new", k_new, None, None, None)
    total_new, H_kv, d = k_new.shape
    dev = k_new.get_device()
    vs, vh = _packed(torch, "v_new", v_new, H_kv, d, dev)
    if v_new.shape[0] != total_new:
        raise ValueError("k_new and v_new must have the same shape")
    B, n, size, width, kp, vp, _, table = _pages(torch, k_pages, v_pages, block_table, H_kv, d,
                                                 dev)
    first = _ints(torch, "starts", starts, B, dev)
    total, idx, cu = total_new, None, None
    if index is not None:
        total = index.numel() if isinstance(index, torch.Tensor) else 0
        idx = _ints(torch, "index", index, total, dev)
    if cu_seqlens is not None:
        cu = _ints(torch, "cu_seqlens", cu_seqlens, B + 1, dev)
    elif B == 0 or total % B:
        raise ValueError("without cu_seqlens every row has the same number of entries")
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_paged_append(
        k_pages.data_ptr(), v_pages.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), cu, first, idx,
        table, B, H_kv, d, total, total_new, n, size, width, ks, kh, vs, vh, kp,
        vp, _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_paged_append")
    if stream is not None:
        _in_use(torch, dev, stream, k_pages, v_pages, k_new, v_new, block_table, starts, cu_seqlens,
                index)


def paged_attention(q, k_pages, v_pages, block_table, kv_lens, *, cu_seqlens=None,
                    max_tokens: int | None = None, max_keys: int | None = None,
                    causal: bool = True, scale: float | None = None, out=None, lse=None,
                    stream=None, workspace=None):
    """Attention of new tokens over pages (as paged_append) that hold them already: row b has
    kv_lens[b] keys (int32 [B]), the last of them those of its T tokens in q [total,H_q,d] (prefix
    sums cu_seqlens int32 [B+1]; None: total / B per row). Token t sees the keys
    j <= kv_lens[b] - T + t (causal) or all of them. A call may mix single tokens, drafted tokens in
    a line and chunks of prompts. max_tokens bounds T; it is needed with cu_seqlens, whose values
    stay on the device. max_keys bounds kv_lens (None: what the table holds); up to 640 saves a
    kernel.

    Returns (o [total,H_q,d] bf16, lse [total,H_q] fp32). ``workspace``: a uint8 CUDA tensor of
    gqa_attn_paged_attention_workspace_size bytes that no overlapping call uses; by default one is
    allocated for the call. ``stream`` as prefill_packed."""
    import torch

    qs, qh = _packed(torch, "q", q, None, None, None)
    total, H_q, d = q.shape
    dev = q.get_device()
    B, n, size, width, kp, vp, H_kv, table = _pages(torch, k_pages, v_pages, block_table, None,
                                                    d, dev)
    lens = _ints(torch, "kv_lens", kv_lens, B, dev)
    cu = None
    if cu_seqlens is not None:
        cu = _ints(torch, "cu_seqlens", cu_seqlens, B + 1, dev)
        if max_tokens is None:
            raise ValueError("max_tokens is needed with cu_seqlens")
    else:
        if B == 0 or total % B:
            raise ValueError("without cu_seqlens every row has total / B tokens")
        max_tokens = max(1, total // B) if max_tokens is None else max_tokens
    if max_keys is not None and max_keys < 1:
        raise ValueError("max_keys must be positive")
    out, lse = _outputs(torch, q, out, lse, stream)
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    given = workspace
    if workspace is None:
        # from the launch stream's pool: its memory is reused only behind this call
        workspace = _empty(torch, q, _paged_workspace(H_q, H_kv, d, max_tokens), torch.uint8,
                           stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on cuda:{dev}")
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_paged_attention(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), lse.data_ptr(), cu,
        lens, table, B, H_q, H_kv, d, total, max_tokens, max_keys or 0, n, size,
        width, qs, qh, kp, vp, 1 if causal else 0, sc, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_paged_attention")
    if stream is not None:
        _in_use(torch, dev, stream, q, k_pages, v_pages, out, lse, block_table, kv_lens, cu_seqlens,
                given)
    return out, lse


def verify_drafts(target_probs, draft_tokens, u_accept, u_sample, cu_seqlens=None, *,
                  draft_probs=None, accepted=None, next_tokens=None, stream=None):
    """Which drafted tokens stand, and the token that follows them (speculative sampling). Row b's
    drafted tokens are packed in draft_tokens (int32 [total]; prefix sums cu_seqlens int32 [B+1],
    None: total / B per row), their draft distributions in draft_probs [total,V] float32 (None: each
    draft was certain), the target's in target_probs [total + B,V] float32, n + 1 for a row of n
    drafts. Draft i stands if u_accept[i] * q(x) < p(x) (float32 [total], from [0, 1)) and all
    before it stand; the next token is drawn with u_sample (float32 [B]) from max(p - q, 0) where
    the first one falls, or from the last p, as the lowest token whose cumulative sum is above
    u_sample times the sum.

    Returns (accepted, next_tokens), int32 [B]. ``stream`` as prefill_packed."""
    import torch

    def table(name, t):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not torch.float32:
            raise TypeError(f"{name} must be a float32 CUDA tensor")
        if t.dim() != 2:
            raise ValueError("target_probs and draft_probs must be [rows, V]")
        n, V = t.shape
        st, sv = t.stride()
        if sv != 1 and V > 1:
            raise ValueError(f"the last dimension of {name} must be contiguous")
        return n, V, st

    rows, V, target_stride = table("target_probs", target_probs)
    dev = target_probs.get_device()
    q_ptr, draft_stride = None, V
    if draft_probs is not None:
        n_q, V_q, draft_stride = table("draft_probs", draft_probs)
        if V_q != V:
            raise ValueError("target_probs and draft_probs must be [rows, V]")
        q_ptr = draft_probs.data_ptr()
    total = draft_tokens.numel() if isinstance(draft_tokens, torch.Tensor) else 0
    toks = _ints(torch, "draft_tokens", draft_tokens, total, dev)
    B = rows - total
    if B < 0:
        raise ValueError("target_probs must have a row for every drafted token and one per row")
    ua = _floats(torch, "u_accept", u_accept, total, dev)
    us = _floats(torch, "u_sample", u_sample, B, dev)
    cu = None
    if cu_seqlens is not None:
        cu = _ints(torch, "cu_seqlens", cu_seqlens, B + 1, dev)
    elif B == 0 or total % B:
        raise ValueError("without cu_seqlens every row has the same number of drafted tokens")
    if draft_probs is not None and (n_q != total or draft_probs.get_device() != dev):
        raise ValueError(f"draft_probs must have {total} rows and be on cuda:{dev}")
    accepted = (_empty(torch, target_probs, B, torch.int32, stream) if accepted is None
                else _counts(torch, "accepted", target_probs, accepted, B))
    next_tokens = (_empty(torch, target_probs, B, torch.int32, stream) if next_tokens is None
                   else _counts(torch, "next_tokens", target_probs, next_tokens, B))
    rc = _on_device(torch, dev, lambda: lib().gqa_attn_verify_drafts(
        target_probs.data_ptr(), q_ptr, toks, ua, us, cu, accepted.data_ptr(),
        next_tokens.data_ptr(), B, total, V, target_stride, draft_stride,
        _raw_stream(torch, dev, stream)))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_verify_drafts")
    if stream is not None:
        _in_use(torch, dev, stream, target_probs, draft_probs, draft_tokens, u_accept, u_sample,
                cu_seqlens, accepted, next_tokens)
    return accepted, next_tokens


def check(stream=None):
    """Synchronises the stream and raises if the device status word is set."""
    rc = gqa_attn_check(_stream_ptr(stream))
    if rc != GQA_OK:
        raise GqaError(rc, "gqa_attn_check")
