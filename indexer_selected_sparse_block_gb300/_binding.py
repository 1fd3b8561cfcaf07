"""ctypes binding of libsfa (the C ABI in include/sfa.h).

Argument marshalling only: every step of the method runs in libsfa's CUDA kernels.  Tensors
are torch CUDA tensors (torch provides device memory and streams); each function passes
their raw pointers, sizes and the current stream to the C entry point of the same name and
raises ``SfaError`` on a non-zero status.  There is no CPU fallback: if libsfa.so is not
built, the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsfa.so")

SFA_OK, SFA_ERR_INVALID_ARG, SFA_ERR_UNSUPPORTED, SFA_ERR_CUDA, SFA_ERR_WORKSPACE = range(5)
SFA_BF16, SFA_F32, SFA_Q8_0 = 0, 1, 2
SFA_DEV_BAD_BLOCK, SFA_DEV_BAD_NSEL, SFA_DEV_BAD_QUERY, SFA_DEV_TIMEOUT = 1, 2, 4, 8
SFA_DEV_BAD_CELL, SFA_DEV_FP16_RANGE = 16, 32
SFA_DEV_BAD_LENGTH, SFA_DEV_NO_PAGES, SFA_DEV_BAD_TREE = 64, 128, 256
SFA_PART_ALL, SFA_PART_SELECTED, SFA_PART_WINDOW, SFA_PART_DRAFTED = 0, 1, 2, 3
SFA_REFINE_MAX_BLOCKS = 131072  # longest row sfa_topk_blocks_refine takes

_lib = None
_vp, _i64, _int, _f32, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                              ctypes.c_size_t)
_f64 = ctypes.c_double

class _RowCopy(ctypes.Structure):
    """sfa_row_copy of include/sfa.h."""
    _fields_ = [("dst", ctypes.c_void_p), ("dst_pitch", ctypes.c_int64),
                ("src", ctypes.c_void_p), ("src_pitch", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64), ("n_rows", ctypes.c_int64)]


class _CellWrite(ctypes.Structure):
    """sfa_cell_write of include/sfa.h."""
    _fields_ = [("src", ctypes.c_void_p), ("src_stride", ctypes.c_int64),
                ("dst", ctypes.c_void_p), ("src_dtype", ctypes.c_int),
                ("dst_dtype", ctypes.c_int), ("n_inner", ctypes.c_int), ("d", ctypes.c_int)]


SFA_MAX_ROW_COPIES = 8
SFA_MAX_CELL_WRITES = 4
SFA_MAX_ROT = 512
SFA_MAX_ROTATIONS = 4
SFA_MAX_TREE = 1024

# name -> (restype, argtypes); mirrors include/sfa.h
SIGNATURES = {
    "sfa_pool_index_keys": (_int, [_vp, _int, _i64, _int, _int, _int, _i64, _i64, _vp, _i64, _vp,
                                   _i64, _vp]),
    "sfa_pool_index_keys_transformed": (_int, [_vp, _int, _i64, _int, _int, _int, _i64, _i64,
                                               _int, _vp, _vp, _f32, _int, _f32, _int, _i64,
                                               _vp, _i64, _vp, _i64, _vp]),
    "sfa_pool_index_keys_paged": (_int, [_vp, _int, _i64, _vp, _i64, _int, _int, _int, _i64,
                                         _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "sfa_index_scores": (_int, [_vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _vp, _i64,
                                _int, _i64, _vp, _i64, _vp, _vp]),
    "sfa_index_scores_bounded": (_int, [_vp, _vp, _vp, _vp, _int, _int, _int, _int, _int, _vp,
                                        _i64, _vp, _i64, _int, _i64, _vp, _vp, _i64, _vp, _vp]),
    "sfa_quantize_pooled_keys_i8": (_int, [_vp, _i64, _int, _int, _i64, _i64, _vp, _i64, _vp,
                                           _i64, _vp]),
    "sfa_index_scores_bounded_i8": (_int, [_vp, _vp, _vp, _vp, _int, _int, _int, _int, _vp, _i64,
                                           _vp, _i64, _int, _i64, _vp, _vp, _i64, _vp, _vp]),
    "sfa_topk_workspace_bytes": (_sz, [_int, _i64, _int]),
    "sfa_attend_plan": (_int, [_int, _int, _int, _int, _int, _i64, _int, _int, _vp, _vp]),
    "sfa_topk_refine_workspace_bytes": (_sz, [_int, _i64]),
    "sfa_topk_blocks_refine": (_int, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _int, _int, _int, _vp,
                                      _i64, _int, _int, _int, _i64, _vp, _vp, _vp, _sz, _vp,
                                      _vp]),
    "sfa_topk_blocks": (_int, [_vp, _i64, _vp, _int, _int, _int, _i64, _vp, _vp, _vp, _sz, _vp,
                               _vp]),
    "sfa_attend_workspace_bytes": (_sz, [_int, _int, _int, _int, _i64]),
    "sfa_gather_attend": (_int, [_vp, _vp, _vp, _int, _int, _i64, _int, _int, _int, _int, _int,
                                 _f32, _vp, _vp, _vp, _vp, _int, _int, _vp, _vp, _vp, _sz, _vp,
                                 _vp]),
    "sfa_dense_attend": (_int, [_vp, _vp, _vp, _int, _int, _i64, _int, _int, _int, _int, _int,
                                _f32, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp, _vp]),
    "sfa_window_kv_max": (_i64, [_int, _int, _i64, _int]),
    "sfa_gather_attend_window": (_int, [_vp, _vp, _vp, _int, _int, _i64, _int, _int, _int, _int,
                                        _int, _f32, _vp, _vp, _vp, _vp, _int, _int, _i64, _int,
                                        _vp, _vp, _vp, _sz, _vp, _vp]),
    "sfa_combine_attention": (_int, [_vp, _vp, _vp, _vp, _i64, _int, _vp, _vp, _vp]),
    "sfa_gather_kv_bandwidth": (_int, [_vp, _vp, _int, _i64, _int, _int, _int, _int, _vp, _vp, _vp,
                                       _vp, _int, _int, _vp, _vp, _vp]),
    "sfa_gather_attend_noalloc": (_int, [_vp, _vp, _vp, _int, _int, _i64, _int, _int, _int,
                                         _int, _int, _f32, _vp, _vp, _vp, _vp, _int, _int, _vp,
                                         _vp, _vp, _vp]),
    "sfa_gather_attend_paged": (_int, [_vp, _vp, _vp, _int, _i64, _vp, _int, _i64, _int, _int,
                                       _int, _int, _int, _f32, _vp, _vp, _vp, _vp, _int, _int,
                                       _vp, _vp, _vp, _sz, _vp, _vp]),
    "sfa_dense_attend_paged": (_int, [_vp, _vp, _vp, _int, _i64, _vp, _int, _i64, _int, _int,
                                      _int, _int, _int, _f32, _vp, _vp, _i64, _vp, _vp, _vp, _sz,
                                      _vp, _vp]),
    "sfa_q8_0_row_bytes": (_sz, [_int]),
    "sfa_quantize_kv_q8_0": (_int, [_vp, _int, _i64, _i64, _int, _i64, _vp, _i64, _vp, _vp]),
    "sfa_copy_cache_rows": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _vp]),
    "sfa_copy_cache_rows_multi": (_int, [_int, _vp, _vp]),
    "sfa_build_page_maps": (_int, [_vp, _vp, _int, _int, _vp, _i64, _vp, _int, _vp, _i64, _vp,
                                   _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp]),
    "sfa_write_cells": (_int, [_int, _vp, _vp, _i64, _i64, _vp, _vp]),
    "sfa_chunk_attend_workspace_bytes": (_sz, [_int, _int, _int, _int, _int, _int, _int, _int,
                                               _int, _i64, _int]),
    "sfa_chunk_attend_paged": (_int, [_vp, _vp, _vp, _int, _i64, _vp, _i64, _int, _int, _int,
                                      _int, _int, _int, _int, _f32, _vp, _vp, _int, _i64, _vp,
                                      _int, _vp, _vp, _sz, _vp, _vp]),
    "sfa_rope_frequencies": (_int, [_int, _f64, _f64, _f64, _f64, _f64, _vp]),
    "sfa_rope_init": (_int, [_vp, _int, _int, _vp, _f64]),
    "sfa_rotate_rows": (_int, [_int, _vp, _vp, _int, _vp, _i64, _vp, _i64, _vp, _vp]),
    "sfa_tree_attend_workspace_bytes": (_sz, [_int, _int, _int, _int, _int, _int, _int, _int, _int,
                                              _int, _i64, _int]),
    "sfa_tree_attend_paged": (_int, [_vp, _vp, _vp, _int, _i64, _vp, _i64, _int, _int, _int, _int, _int,
                                     _int, _int, _f32, _vp, _vp, _vp, _int, _int, _int, _i64, _vp, _int,
                                     _vp, _vp, _sz, _vp, _vp]),
    "sfa_build_tree_maps": (_int, [_vp, _vp, _vp, _int, _i64, _vp, _int, _vp, _vp, _vp, _vp]),
    "sfa_tree_accept": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "sfa_tree_commit": (_int, [_int, _vp, _i64, _vp, _vp, _vp, _int, _i64, _vp, _i64, _vp, _int, _vp,
                               _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp]),
    "sfa_read_device_status": (_int, [_vp, _vp, _vp]),
    "sfa_status_string": (ctypes.c_char_p, [_int]),
}


class SfaError(RuntimeError):
    """A non-zero status returned by libsfa."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {lib().sfa_status_string(status).decode()}")


def lib(path: str | None = None):
    """Loads libsfa.so (built by ``__graft_entry__.build()``); raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libsfa.so is not built ({p}); run __graft_entry__.build() first")
    L = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    if path is None:
        _lib = L
    return L


def _p(t, strided=False):
    """Device pointer of t; strided=True when the caller passes t's strides to the library."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libsfa takes CUDA tensors only")
    if not strided and not t.is_contiguous():
        raise ValueError("libsfa takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _p_out(t):
    """Pointer of an attention output: a CUDA tensor, or a page-locked host tensor that the
    device writes directly."""
    if t is not None and not t.is_cuda:
        if not t.is_pinned():
            raise ValueError("an attention output on the host must be in page-locked memory")
        if not t.is_contiguous():
            raise ValueError("libsfa takes contiguous tensors only")
        return ctypes.c_void_p(t.data_ptr())
    return _p(t)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _scratch(n_bytes, device, stream):
    """A workspace for one call on `stream` (None: the current one).  It comes from that stream's
    own pool: a block of another stream's may still be in use there, by work that this stream does
    not wait for, and this one could be handed out there while the call still runs."""
    if stream is None:
        return torch.empty(n_bytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n_bytes, dtype=torch.uint8, device=device)


def _check(fn: str, rc: int):
    if rc != SFA_OK:
        raise SfaError(fn, rc)


def _dtype_code(t) -> int:
    if t.dtype == torch.bfloat16:
        return SFA_BF16
    if t.dtype == torch.float32:
        return SFA_F32
    if t.dtype == torch.uint8:   # q8_0 cache rows
        return SFA_Q8_0
    raise ValueError(f"unsupported dtype {t.dtype}")


def kbar_shape(n_seq: int, blk_cap: int, d_idx: int):
    """Shape of the pooled-key table: [n_seq][blk_cap][2*d_idx] bf16 (hi, lo halves)."""
    return (n_seq, blk_cap, 2 * d_idx)


def sfa_pool_index_keys(X, compress_ratio: int, blk_begin: int, blk_end: int, Kbar,
                        Kbar_r=None, stream=None):
    """X [n_seq][n_tok_cap][d_idx] (bf16/f32) -> rows [blk_begin, blk_end) of Kbar, and of the
    bound factors Kbar_r [n_seq][blk_cap] fp32 when given."""
    n_seq, _, d_idx = X.shape
    rc = lib().sfa_pool_index_keys(_p(X), _dtype_code(X), X.stride(0), n_seq, d_idx,
                                   compress_ratio, blk_begin, blk_end, _p(Kbar), Kbar.stride(0),
                                   _p(Kbar_r), Kbar_r.stride(0) if Kbar_r is not None else 0,
                                   _stream(stream))
    _check("sfa_pool_index_keys", rc)


def sfa_pool_index_keys_transformed(X, compress_ratio: int, blk_begin: int, blk_end: int, Kbar,
                                    Kbar_r=None, *, norm: int = 0, gamma=None, beta=None,
                                    eps: float = 1e-6, n_rot: int = 0, rope_base: float = 10000.0,
                                    rope_neox: bool = True, pos_offset: int = 0, stream=None):
    """sfa_pool_index_keys with the pooled key normalised (norm 0 none, 1 RMS, 2 layer; gamma,
    beta [d_idx] fp32 on the device) and its first n_rot dims rotated at b*cr + pos_offset."""
    n_seq, _, d_idx = X.shape
    rc = lib().sfa_pool_index_keys_transformed(
        _p(X), _dtype_code(X), X.stride(0), n_seq, d_idx, compress_ratio, blk_begin, blk_end,
        norm, _p(gamma), _p(beta), eps, n_rot, rope_base, int(rope_neox), pos_offset, _p(Kbar),
        Kbar.stride(0), _p(Kbar_r), Kbar_r.stride(0) if Kbar_r is not None else 0,
        _stream(stream))
    _check("sfa_pool_index_keys_transformed", rc)


def sfa_index_scores(q_idx, w, q_seq, q_pos, Kbar, compress_ratio: int, n_blk_max: int, scores,
                     q_group: int = 1, dev_status=None, stream=None):
    """scores[i][b] = sum_j w[i][j] * relu(q_idx[i][j] . kbar_b) for b < B_i."""
    n_q, h_idx, d_idx = q_idx.shape
    rc = lib().sfa_index_scores(_p(q_idx), _p(w), _p(q_seq), _p(q_pos), n_q, q_group, h_idx,
                                d_idx, compress_ratio, _p(Kbar), Kbar.stride(0), Kbar.shape[0],
                                n_blk_max, _p(scores), scores.stride(0), _p(dev_status),
                                _stream(stream))
    _check("sfa_index_scores", rc)


def sfa_index_scores_bounded(q_idx, w, q_seq, q_pos, Kbar, Kbar_r, compress_ratio: int,
                             n_blk_max: int, lower, upper, q_group: int = 1, dev_status=None,
                             stream=None):
    """lower[i][b] <= s_ib <= upper[i][b] for the hi + lo score s_ib, from the hi halves of the
    pooled keys and their bound factors Kbar_r only."""
    n_q, h_idx, d_idx = q_idx.shape
    if lower.stride(0) != upper.stride(0):
        raise ValueError("lower and upper must share a row stride")
    rc = lib().sfa_index_scores_bounded(_p(q_idx), _p(w), _p(q_seq), _p(q_pos), n_q, q_group,
                                        h_idx, d_idx, compress_ratio, _p(Kbar), Kbar.stride(0),
                                        _p(Kbar_r), Kbar_r.stride(0), Kbar.shape[0], n_blk_max,
                                        _p(lower), _p(upper), lower.stride(0), _p(dev_status),
                                        _stream(stream))
    _check("sfa_index_scores_bounded", rc)


def k8_shapes(n_seq: int, blk_cap: int, d_idx: int):
    """Shapes of the 8-bit pooled-key copy: codes [n_seq][blk_cap][d_idx] (int8 storage of the
    bytes c + 128) and (scale, bound factor) pairs [n_seq][blk_cap][2] fp32."""
    return (n_seq, blk_cap, d_idx), (n_seq, blk_cap, 2)


def sfa_quantize_pooled_keys_i8(Kbar, blk_begin: int, blk_end: int, K8, K8_sr, stream=None):
    """Rows [blk_begin, blk_end) of the 8-bit copy (K8 codes, K8_sr scale and bound factor) of
    the pooled keys m = hi + lo in Kbar."""
    n_seq, _, two_d = Kbar.shape
    if K8.dtype != torch.int8 or K8_sr.dtype != torch.float32:
        raise ValueError("K8 must be int8 and K8_sr float32")
    rc = lib().sfa_quantize_pooled_keys_i8(_p(Kbar), Kbar.stride(0), n_seq, two_d // 2,
                                           blk_begin, blk_end, _p(K8), K8.stride(0), _p(K8_sr),
                                           K8_sr.stride(0), _stream(stream))
    _check("sfa_quantize_pooled_keys_i8", rc)


def sfa_index_scores_bounded_i8(q_idx, w, q_seq, q_pos, K8, K8_sr, compress_ratio: int,
                                n_blk_max: int, lower, upper, dev_status=None, stream=None):
    """lower[i][b] <= s_ib <= upper[i][b] for the hi + lo score s_ib, from the 8-bit copy of the
    pooled keys (sfa_quantize_pooled_keys_i8)."""
    n_q, h_idx, d_idx = q_idx.shape
    if lower.stride(0) != upper.stride(0):
        raise ValueError("lower and upper must share a row stride")
    rc = lib().sfa_index_scores_bounded_i8(_p(q_idx), _p(w), _p(q_seq), _p(q_pos), n_q, h_idx,
                                           d_idx, compress_ratio, _p(K8), K8.stride(0),
                                           _p(K8_sr), K8_sr.stride(0), K8.shape[0], n_blk_max,
                                           _p(lower), _p(upper), lower.stride(0),
                                           _p(dev_status), _stream(stream))
    _check("sfa_index_scores_bounded_i8", rc)


def sfa_topk_refine_workspace_bytes(n_q: int, n_blk_max: int) -> int:
    return int(lib().sfa_topk_refine_workspace_bytes(n_q, n_blk_max))


def sfa_topk_blocks_refine(lower, upper, q_idx, w, q_seq, q_pos, Kbar, compress_ratio: int,
                           top_k: int, n_blk_max: int, blk_idx, n_sel, workspace=None,
                           dev_status=None, stream=None):
    """The top_k best blocks by the hi + lo score, from its lower and upper bounds: only the
    blocks the bounds cannot rule out are rescored."""
    n_q, h_idx, d_idx = q_idx.shape
    need = sfa_topk_refine_workspace_bytes(n_q, n_blk_max)
    if workspace is None:
        workspace = _scratch(max(need, 16), q_pos.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().sfa_topk_blocks_refine(_p(lower), _p(upper), lower.stride(0), _p(q_idx), _p(w),
                                      _p(q_seq), _p(q_pos), n_q, h_idx, d_idx, _p(Kbar),
                                      Kbar.stride(0), Kbar.shape[0], compress_ratio, top_k,
                                      n_blk_max, _p(blk_idx), _p(n_sel), _p(workspace),
                                      ws_bytes, _p(dev_status), _stream(stream))
    _check("sfa_topk_blocks_refine", rc)


def sfa_topk_workspace_bytes(n_q: int, n_blk_max: int, top_k: int) -> int:
    return int(lib().sfa_topk_workspace_bytes(n_q, n_blk_max, top_k))


def sfa_topk_blocks(scores, q_pos, compress_ratio: int, top_k: int, n_blk_max: int, blk_idx,
                    n_sel, workspace=None, dev_status=None, stream=None):
    """The top_k best blocks of each query (ascending, -1 padded) and their count.  scores may
    be a view whose rows are apart (score_stride = scores.stride(0)); each row contiguous."""
    if scores.dim() != 2 or scores.stride(1) != 1:
        raise ValueError("scores must be [n_q][>= n_blk_max] with contiguous rows")
    n_q = q_pos.shape[0]
    need = sfa_topk_workspace_bytes(n_q, n_blk_max, top_k)
    if need and workspace is None:
        workspace = _scratch(need, q_pos.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sfa_topk_blocks(_p(scores, strided=True), scores.stride(0), _p(q_pos), n_q,
                               compress_ratio,
                               top_k, n_blk_max, _p(blk_idx), _p(n_sel), _p(workspace),
                               ws_bytes, _p(dev_status), _stream(stream))
    _check("sfa_topk_blocks", rc)


def sfa_attend_workspace_bytes(n_q: int, h_q: int, h_kv: int, dv: int, n_kv_max: int) -> int:
    return int(lib().sfa_attend_workspace_bytes(n_q, h_q, h_kv, dv, n_kv_max))


def sfa_attend_plan(dtype_code: int, n_q: int, h_kv: int, dkq: int, has_v: bool, n_kv_max: int,
                    compress_ratio: int, dense: bool = False):
    """(n_split, kernels): CTAs per (query, KV head) list and kernels one attention call
    launches on the current device."""
    ns, nk = ctypes.c_int(0), ctypes.c_int(0)
    rc = lib().sfa_attend_plan(dtype_code, n_q, h_kv, dkq, int(has_v), n_kv_max, compress_ratio,
                               int(dense), ctypes.byref(ns), ctypes.byref(nk))
    _check("sfa_attend_plan", rc)
    return ns.value, nk.value


def _check_qkv(Q, K, V):
    if V is not None and K.dtype != V.dtype:
        raise ValueError("K and V must share a dtype")
    if K.dtype == torch.uint8:   # q8_0 cache rows: Q stays bf16
        if Q.dtype != torch.bfloat16:
            raise ValueError("a q8_0 cache takes a bf16 Q")
    elif Q.dtype != K.dtype:
        raise ValueError("Q and K must share a dtype")


def _attn_dims(Q, K, V, O):
    n_q, h_q, dkq = Q.shape
    n_seq, n_tok_cap, h_kv, _ = K.shape
    dv = O.shape[-1]
    _check_qkv(Q, K, V)
    return n_q, h_q, dkq, n_seq, n_tok_cap, h_kv, dv


def sfa_gather_attend(Q, K, V, q_seq, q_pos, blk_idx, n_sel, top_k: int, compress_ratio: int,
                      scale: float, O, lse=None, workspace=None, dev_status=None, stream=None):
    """Attention of each query over its kept blocks plus its tail."""
    n_q, h_q, dkq, n_seq, n_tok_cap, h_kv, dv = _attn_dims(Q, K, V, O)
    n_kv_max = top_k * compress_ratio + compress_ratio - 1
    need = sfa_attend_workspace_bytes(n_q, h_q, h_kv, dv, n_kv_max)
    if need and workspace is None:
        workspace = _scratch(need, Q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sfa_gather_attend(_p(Q), _p(K), _p(V), _dtype_code(K), n_seq, n_tok_cap, n_q, h_q,
                                 h_kv, dkq, dv, float(scale), _p(q_seq), _p(q_pos), _p(blk_idx),
                                 _p(n_sel), top_k, compress_ratio, _p_out(O), _p_out(lse),
                                 _p(workspace), ws_bytes, _p(dev_status), _stream(stream))
    _check("sfa_gather_attend", rc)


def sfa_window_kv_max(top_k: int, compress_ratio: int, window: int, part: int = 0) -> int:
    return int(lib().sfa_window_kv_max(top_k, compress_ratio, window, part))


def sfa_gather_attend_window(Q, K, V, q_seq, q_pos, blk_idx, n_sel, top_k: int,
                             compress_ratio: int, window: int, scale: float, O, lse=None,
                             part: int = SFA_PART_ALL, workspace=None, dev_status=None,
                             stream=None):
    """Attention over the kept blocks, the tail and a dense window of the `window` most recent
    positions (part: the whole set, its kept part before the window, or the window suffix)."""
    n_q, h_q, dkq, n_seq, n_tok_cap, h_kv, dv = _attn_dims(Q, K, V, O)
    n_kv_max = sfa_window_kv_max(top_k, compress_ratio, window, part)
    need = sfa_attend_workspace_bytes(n_q, h_q, h_kv, dv, n_kv_max)
    if need and workspace is None:
        workspace = _scratch(need, Q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sfa_gather_attend_window(_p(Q), _p(K), _p(V), _dtype_code(K), n_seq, n_tok_cap,
                                        n_q, h_q, h_kv, dkq, dv, float(scale), _p(q_seq),
                                        _p(q_pos), _p(blk_idx), _p(n_sel), top_k,
                                        compress_ratio, int(window), int(part), _p_out(O),
                                        _p_out(lse), _p(workspace), ws_bytes, _p(dev_status),
                                        _stream(stream))
    _check("sfa_gather_attend_window", rc)


def sfa_combine_attention(O_a, lse_a, O_b, lse_b, O, lse, stream=None):
    """O, lse = the attention over the union of two disjoint key sets, from each set's (O, lse)
    ([rows][dv] and [rows] fp32; O / lse may be either input)."""
    dv = O.shape[-1]
    n_rows = O.numel() // dv
    for t in (O_a, O_b, O):
        if t.numel() != n_rows * dv or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError("O_a, O_b, O must be contiguous fp32 tensors of one shape")
    for t in (lse_a, lse_b, lse):
        if t.numel() != n_rows or not t.is_contiguous() or t.dtype != torch.float32:
            raise ValueError("lse_a, lse_b, lse must be contiguous fp32 tensors of O's rows")
    rc = lib().sfa_combine_attention(_p(O_a), _p(lse_a), _p(O_b), _p(lse_b), n_rows, dv, _p_out(O),
                                     _p_out(lse), _stream(stream))
    _check("sfa_combine_attention", rc)


def sfa_gather_kv_bandwidth(K, V, q_seq, q_pos, blk_idx, n_sel, top_k: int, compress_ratio: int,
                            dkq: int, dv: int, checksum, dev_status=None, stream=None):
    """A measurement: the K/V rows sfa_gather_attend would attend, moved into shared memory
    and nothing else (its time is the attention's data-movement ceiling on these lists)."""
    n_seq, n_tok_cap, h_kv = K.shape[0], K.shape[1], K.shape[2]
    rc = lib().sfa_gather_kv_bandwidth(_p(K), _p(V), n_seq, n_tok_cap, q_seq.numel(), h_kv, dkq,
                                       dv, _p(q_seq), _p(q_pos), _p(blk_idx), _p(n_sel), top_k,
                                       compress_ratio, _p(checksum), _p(dev_status),
                                       _stream(stream))
    _check("sfa_gather_kv_bandwidth", rc)


def sfa_gather_attend_noalloc(Q, K, V, q_seq, q_pos, blk_idx, n_sel, top_k: int,
                              compress_ratio: int, scale: float, O, lse=None, dev_status=None,
                              stream=None):
    """sfa_gather_attend without a workspace: for callers that cannot allocate device memory
    when they call (their split-KV scratch is a fixed 16 MiB array inside libsfa, shared by
    every call on the device; overlapping calls on the GPU race on it)."""
    n_q, h_q, dkq, n_seq, n_tok_cap, h_kv, dv = _attn_dims(Q, K, V, O)
    rc = lib().sfa_gather_attend_noalloc(_p(Q), _p(K), _p(V), _dtype_code(K), n_seq, n_tok_cap,
                                         n_q, h_q, h_kv, dkq, dv, float(scale), _p(q_seq),
                                         _p(q_pos), _p(blk_idx), _p(n_sel), top_k,
                                         compress_ratio, _p_out(O), _p_out(lse), _p(dev_status),
                                         _stream(stream))
    _check("sfa_gather_attend_noalloc", rc)


def sfa_dense_attend(Q, K, V, q_seq, q_pos, n_kv_max: int, scale: float, O, lse=None,
                     workspace=None, dev_status=None, stream=None):
    """Causal attention of each query over all of its sequence's tokens 0..p_i."""
    n_q, h_q, dkq, n_seq, n_tok_cap, h_kv, dv = _attn_dims(Q, K, V, O)
    need = sfa_attend_workspace_bytes(n_q, h_q, h_kv, dv, n_kv_max)
    if need and workspace is None:
        workspace = _scratch(need, Q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sfa_dense_attend(_p(Q), _p(K), _p(V), _dtype_code(K), n_seq, n_tok_cap, n_q, h_q,
                                h_kv, dkq, dv, float(scale), _p(q_seq), _p(q_pos), n_kv_max,
                                _p_out(O), _p_out(lse), _p(workspace), ws_bytes, _p(dev_status),
                                _stream(stream))
    _check("sfa_dense_attend", rc)


def _paged_dims(cell_of, n_cells_of):
    if cell_of.dtype != torch.int32 or cell_of.dim() != 2 or not cell_of.is_contiguous():
        raise ValueError("cell_of must be a contiguous [n_seq][n_pos_cap] int32 tensor")
    return cell_of.shape[0], cell_of.shape[1], n_cells_of


def sfa_pool_index_keys_paged(X, cell_of, compress_ratio: int, blk_begin: int, blk_end: int, Kbar,
                              Kbar_r=None, dev_status=None, stream=None):
    """Paged layout: X [n_cells][d_idx] raw index keys, one cell per row; position t of
    sequence s is in cell cell_of[s][t].  Writes rows [blk_begin, blk_end) of Kbar (and Kbar_r)
    as sfa_pool_index_keys does for the gathered layout."""
    n_cells, d_idx = X.shape
    n_seq, n_pos_cap, _ = _paged_dims(cell_of, n_cells)
    rc = lib().sfa_pool_index_keys_paged(_p(X), _dtype_code(X), n_cells, _p(cell_of), n_pos_cap,
                                         n_seq, d_idx, compress_ratio, blk_begin, blk_end,
                                         _p(Kbar), Kbar.stride(0), _p(Kbar_r),
                                         Kbar_r.stride(0) if Kbar_r is not None else 0,
                                         _p(dev_status), _stream(stream))
    _check("sfa_pool_index_keys_paged", rc)


def _paged_attn_dims(Q, K, V, O, cell_of):
    n_q, h_q, dkq = Q.shape
    n_cells, h_kv, _ = K.shape
    if V is not None and V.shape[0] != n_cells:
        raise ValueError("V must have K's cell count")
    _check_qkv(Q, K, V)
    n_seq, n_pos_cap, _ = _paged_dims(cell_of, n_cells)
    return n_q, h_q, dkq, n_cells, n_seq, n_pos_cap, h_kv, O.shape[-1]


def sfa_gather_attend_paged(Q, K, V, cell_of, q_seq, q_pos, blk_idx, n_sel, top_k: int,
                            compress_ratio: int, scale: float, O, lse=None, workspace=None,
                            dev_status=None, stream=None):
    """sfa_gather_attend on the paged layout: K [n_cells][h_kv][dkq], V [n_cells][h_kv][dv] or
    None, position t of sequence s in cell cell_of[s][t]."""
    n_q, h_q, dkq, n_cells, n_seq, n_pos_cap, h_kv, dv = _paged_attn_dims(Q, K, V, O, cell_of)
    n_kv_max = top_k * compress_ratio + compress_ratio - 1
    need = sfa_attend_workspace_bytes(n_q, h_q, h_kv, dv, n_kv_max)
    if need and workspace is None:
        workspace = _scratch(need, Q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sfa_gather_attend_paged(_p(Q), _p(K), _p(V), _dtype_code(K), n_cells, _p(cell_of),
                                       n_seq, n_pos_cap, n_q, h_q, h_kv, dkq, dv, float(scale),
                                       _p(q_seq), _p(q_pos), _p(blk_idx), _p(n_sel), top_k,
                                       compress_ratio, _p_out(O), _p_out(lse), _p(workspace),
                                       ws_bytes, _p(dev_status), _stream(stream))
    _check("sfa_gather_attend_paged", rc)


def sfa_dense_attend_paged(Q, K, V, cell_of, q_seq, q_pos, n_kv_max: int, scale: float, O,
                           lse=None, workspace=None, dev_status=None, stream=None):
    """sfa_dense_attend on the paged layout (see sfa_gather_attend_paged)."""
    n_q, h_q, dkq, n_cells, n_seq, n_pos_cap, h_kv, dv = _paged_attn_dims(Q, K, V, O, cell_of)
    need = sfa_attend_workspace_bytes(n_q, h_q, h_kv, dv, n_kv_max)
    if need and workspace is None:
        workspace = _scratch(need, Q.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().sfa_dense_attend_paged(_p(Q), _p(K), _p(V), _dtype_code(K), n_cells, _p(cell_of),
                                      n_seq, n_pos_cap, n_q, h_q, h_kv, dkq, dv, float(scale),
                                      _p(q_seq), _p(q_pos), n_kv_max, _p_out(O), _p_out(lse),
                                      _p(workspace), ws_bytes, _p(dev_status), _stream(stream))
    _check("sfa_dense_attend_paged", rc)


def sfa_q8_0_row_bytes(d: int) -> int:
    """Bytes of one q8_0 cache row of d elements (codes, binary16 scales, padding to 16)."""
    return int(lib().sfa_q8_0_row_bytes(d))


def sfa_quantize_kv_q8_0(X, Y, dev_status=None, stream=None):
    """q8_0 rows of X [n_outer][n_inner][d] (bf16/f32) into Y [n_outer][n_inner][row_bytes(d)]
    uint8; within an outer index the rows of both are contiguous (a cache slice of new tokens of
    every sequence viewed as [n_seq][tokens * h_kv][d])."""
    n_outer, n_inner, d = X.shape
    rb = sfa_q8_0_row_bytes(d)
    if Y.dtype != torch.uint8 or tuple(Y.shape) != (n_outer, n_inner, rb):
        raise ValueError(f"Y must be uint8 [{n_outer}][{n_inner}][{rb}]")
    if (X.stride(2), Y.stride(2)) != (1, 1) or (n_inner > 1 and (X.stride(1), Y.stride(1)) != (d, rb)):
        raise ValueError("rows must be contiguous within an outer index")
    rc = lib().sfa_quantize_kv_q8_0(_p(X, strided=True), _dtype_code(X), n_outer, n_inner, d,
                                    X.stride(0), _p(Y, strided=True), Y.stride(0), _p(dev_status),
                                    _stream(stream))
    _check("sfa_quantize_kv_q8_0", rc)


def _row_copy(dst, src):
    if tuple(dst.shape) != tuple(src.shape) or dst.dtype != src.dtype or dst.dim() < 1:
        raise ValueError("dst and src must have the same shape and dtype")
    for t in (dst, src):
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError("sfa_copy_cache_rows takes CUDA or page-locked host tensors")
        if t.shape[0] > 0 and not t[0].is_contiguous():
            raise ValueError("each row must be contiguous")
    es = dst.element_size()
    n = dst.shape[0]
    row = dst[0].numel() * es if n > 0 else 0
    dp = dst.stride(0) * es if n > 1 else max(row, 1)
    sp = src.stride(0) * es if n > 1 else max(row, 1)
    return _RowCopy(dst.data_ptr(), dp, src.data_ptr(), sp, max(row, 1), n if row else 0)


def sfa_copy_cache_rows_multi(pairs, stream=None) -> None:
    """Several (dst, src) row copies as sfa_copy_cache_rows makes them, in one kernel launch on the
    device of the first tensor that is on one."""
    pairs = list(pairs)
    if len(pairs) > SFA_MAX_ROW_COPIES:
        raise ValueError(f"at most {SFA_MAX_ROW_COPIES} copies per call")
    arr = (_RowCopy * max(len(pairs), 1))(*[_row_copy(d, s) for d, s in pairs])
    dev = next((t.get_device() for pair in pairs for t in pair if t.is_cuda), None)
    if dev is None:
        dev = torch.cuda.current_device()
    _call(lib().sfa_copy_cache_rows_multi, dev, stream, len(pairs), ctypes.cast(arr, ctypes.c_void_p))


def sfa_copy_cache_rows(dst, src, stream=None) -> None:
    """Copies the rows of src into the rows of dst (the same shape; dim 0 indexes the rows,
    each row contiguous, rows at any stride): one two-dimensional copy, either side on the
    device or in page-locked host memory.  Typically dst = cache[:, p] for a step's new
    position p of every sequence."""
    if tuple(dst.shape) != tuple(src.shape) or dst.dtype != src.dtype or dst.dim() < 1:
        raise ValueError("dst and src must have the same shape and dtype")
    for t in (dst, src):
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError("sfa_copy_cache_rows takes CUDA or page-locked host tensors")
        if t.shape[0] > 0 and not t[0].is_contiguous():
            raise ValueError("each row must be contiguous")
    es = dst.element_size()
    row = dst[0].numel() * es if dst.shape[0] > 0 else 0
    n = dst.shape[0]
    dp = dst.stride(0) * es if n > 1 else row
    sp = src.stride(0) * es if n > 1 else row
    if n == 0 or row == 0:
        return
    rc = lib().sfa_copy_cache_rows(ctypes.c_void_p(dst.data_ptr()), dp,
                                   ctypes.c_void_p(src.data_ptr()), sp, row, n, _stream(stream))
    _check("sfa_copy_cache_rows", rc)


# The paged-serving calls are made every step on small tensors, where the host's time counts:
# their tensors are checked in one look each, their addresses passed as plain integers.
_I32, _BF16, _F32, _U8 = torch.int32, torch.bfloat16, torch.float32, torch.uint8
_CODES = {_BF16: SFA_BF16, _F32: SFA_F32, _U8: SFA_Q8_0}


def _no_tensor(name, t, dev, what):
    """The error for a tensor that a call cannot take."""
    if not t.is_cuda:
        raise ValueError("libsfa takes CUDA tensors only")
    if t.get_device() != dev:
        raise ValueError(f"tensors on cuda:{dev} and {t.device} in one call")
    raise ValueError(f"{name} must be {what}")


def _device_of(t):
    """Index of t's device, the call's."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("libsfa takes CUDA tensors only")
    return dev


def _ints(name, t, n, dev):
    """Address of t: n contiguous int32 values on device dev."""
    if t.dtype is _I32 and t.numel() == n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _no_tensor(name, t, dev, f"a contiguous int32 tensor of {n} entries")


def _int_rows(name, t, n, dev):
    """Address of t, a contiguous int32 [n][any] matrix on device dev."""
    if (t.dtype is not _I32 or t.dim() != 2 or t.get_device() != dev or not t.is_contiguous()
            or t.size(0) != n):
        _no_tensor(name, t, dev, f"a contiguous int32 [{n}][..] tensor")
    return t.data_ptr()


def _call(fn, dev, stream, *args):
    """The entry point on device dev (the library launches on the current one), on `stream` or the
    device's current stream; raises on an error status."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index == dev:
        raw = stream.cuda_stream
    else:
        raise ValueError(f"a stream of cuda:{stream.device_index} for tensors on cuda:{dev}")
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc:
        raise SfaError(fn.__name__, rc)


def sfa_build_page_maps(len_old, len_new, page_size: int, free_pages, free_head, n_pages: int,
                        page_table, cu_new, len_total, q_seq, q_pos, slot, free_head_out,
                        cell_of=None, dev_status=None, stream=None):
    """One step's bookkeeping of a paged cache on the device: pages from free_pages (from entry
    free_head on) into page_table, the new tokens' sequences, positions and cells (q_seq, q_pos,
    slot: rows past the last token get -1), the packed offsets cu_new [n_seq + 1], len_total, and
    the new positions' entries of the per-position map cell_of [n_seq][n_pos] when given."""
    dev = _device_of(len_old)
    n_seq, n_tok, n_free, n_pos, cells = len_old.numel(), slot.numel(), free_pages.numel(), 0, None
    if cell_of is not None:
        cells, n_pos = _int_rows("cell_of", cell_of, n_seq, dev), cell_of.size(1)
    _call(lib().sfa_build_page_maps, dev, stream, _ints("len_old", len_old, n_seq, dev),
          _ints("len_new", len_new, n_seq, dev), n_seq, page_size,
          _ints("free_pages", free_pages, n_free, dev), n_free, _ints("free_head", free_head, 1, dev),
          n_pages, _int_rows("page_table", page_table, n_seq, dev), page_table.size(1),
          _ints("cu_new", cu_new, n_seq + 1, dev), _ints("len_total", len_total, n_seq, dev),
          _ints("q_seq", q_seq, n_tok, dev), _ints("q_pos", q_pos, n_tok, dev),
          _ints("slot", slot, n_tok, dev), n_tok, cells, n_pos,
          _ints("free_head_out", free_head_out, 1, dev),
          None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


_CELL_WRITE = struct.Struct("@QqQiiii")     # sfa_cell_write of include/sfa.h


def _cell_write(src, dst, n_rows, n_cells, dev):
    st, dt = src.dtype, dst.dtype
    if src.dim() == 2:      # [rows][d]: one inner row
        n, d = src.shape
        h = 1
        ok = src.stride(1) == 1 or d == 1
    elif src.dim() == 3:
        n, h, d = src.shape
        _, sh, sd = src.stride()
        ok = (sd == 1 or d == 1) and (sh == d or h == 1)
    else:
        ok, n, h, d = False, 0, 1, 1
    if not ok or n < n_rows or src.get_device() != dev or (st is not _BF16 and st is not _F32):
        _no_tensor("a write's rows", src, dev, f"bf16 or fp32, [>= {n_rows}][d] or [>= {n_rows}]"
                   "[h][d], each row contiguous")
    row = sfa_q8_0_row_bytes(d) if dt is _U8 else d
    if (dst.get_device() != dev or dt not in _CODES or not dst.is_contiguous() or dst.size(0) != n_cells
            or dst.numel() != n_cells * h * row or dst.size(-1) != row):
        _no_tensor("a write's cache", dst, dev, f"a contiguous [{n_cells}][{h}][{row}] tensor for "
                   "these rows")
    return (src.data_ptr(), src.stride(0) if n > 1 else h * d, dst.data_ptr(), _CODES[st], _CODES[dt], h, d)


def sfa_write_cells(writes, slot, dev_status=None, stream=None):
    """For every (rows, cache) pair of writes, at most SFA_MAX_CELL_WRITES, in one launch: row i
    of rows ([n][d] or [n][h][d], rows at any stride) into cell slot[i] of cache ([n_cells][d] or
    [n_cells][h][d], of the same type, bf16 for fp32 rows, or uint8 q8_0 rows).  Negative slots
    are skipped; the others must differ."""
    writes = list(writes)
    if len(writes) > SFA_MAX_CELL_WRITES:
        raise ValueError(f"at most {SFA_MAX_CELL_WRITES} caches per call")
    dev = _device_of(slot)
    n_rows = slot.numel()
    at = _ints("slot", slot, n_rows, dev)
    if not writes:
        return
    n_cells = writes[0][1].size(0)
    packed = b"".join([_CELL_WRITE.pack(*_cell_write(x, y, n_rows, n_cells, dev)) for x, y in writes])
    _call(lib().sfa_write_cells, dev, stream, len(writes), packed, at, n_rows, n_cells,
          None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


def sfa_chunk_attend_workspace_bytes(dtype_code: int, n_seq: int, n_q: int, h_q: int, h_kv: int,
                                     dkq: int, dv: int, has_v: bool, n_new_max: int, n_kv_max: int,
                                     o_dtype: int = SFA_F32) -> int:
    return int(lib().sfa_chunk_attend_workspace_bytes(dtype_code, n_seq, n_q, h_q, h_kv, dkq, dv,
                                                      int(has_v), n_new_max, n_kv_max, o_dtype))


@functools.lru_cache(maxsize=256)
def _chunk_workspace(dev, *sizes):
    """sfa_chunk_attend_workspace_bytes on device dev: sizes in, a size out."""
    with torch.cuda.device(dev):
        return int(lib().sfa_chunk_attend_workspace_bytes(*sizes))


def sfa_tree_attend_workspace_bytes(dtype_code: int, n_seq: int, n_q: int, h_q: int, h_kv: int, dkq: int,
                                    dv: int, has_v: bool, n_new_max: int, n_kv_max: int,
                                    o_dtype: int = SFA_F32, part: int = SFA_PART_ALL) -> int:
    return int(lib().sfa_tree_attend_workspace_bytes(dtype_code, n_seq, n_q, h_q, h_kv, dkq, dv, int(has_v),
                                                     part, n_new_max, n_kv_max, o_dtype))


@functools.lru_cache(maxsize=256)
def _tree_workspace(dev, part, *sizes):
    """sfa_tree_attend_workspace_bytes on device dev: sizes in, a size out."""
    with torch.cuda.device(dev):
        return int(lib().sfa_tree_attend_workspace_bytes(*sizes[:8], part, *sizes[8:]))


def sfa_chunk_attend_paged(Q, K, V, page_table, page_size: int, cu_new, len_total, n_new_max: int,
                           n_kv_max: int, scale: float, O, lse=None, workspace=None,
                           dev_status=None, stream=None):
    """Causal attention of each sequence's chunk of new tokens (rows cu_new[s] .. cu_new[s + 1] of
    Q [n_q][h_q][dkq]) over its len_total[s] cached tokens, the chunk's own included: K
    [n_cells][h_kv][dkq] and V [n_cells][h_kv][dv] or None, through page_table [n_seq][pages].
    O [n_q][h_q][dv] fp32 or bf16, lse [n_q][h_q] fp32; either may be in page-locked host memory."""
    _attend_pages(None, 0, Q, K, V, page_table, page_size, cu_new, len_total, n_new_max, n_kv_max, scale, O,
                  lse, workspace, dev_status, stream)


def sfa_tree_attend_paged(Q, K, V, page_table, page_size: int, cu_new, len_total, tree_mask, n_new_max: int,
                          n_kv_max: int, scale: float, O, lse=None, part: int = SFA_PART_ALL, workspace=None,
                          dev_status=None, stream=None):
    """Attention of the drafted nodes of each sequence (rows cu_new[s] .. cu_new[s + 1] of Q) over its cached
    tokens and the nodes that their rows of tree_mask [n_q][words] int32 name (sfa_build_tree_maps), or,
    with part SFA_PART_DRAFTED, over those nodes alone.  Otherwise as sfa_chunk_attend_paged."""
    _attend_pages(tree_mask, part, Q, K, V, page_table, page_size, cu_new, len_total, n_new_max, n_kv_max,
                  scale, O, lse, workspace, dev_status, stream)


def _attend_pages(mask, part, Q, K, V, page_table, page_size, cu_new, len_total, n_new_max, n_kv_max, scale, O,
                  lse, workspace, dev_status, stream):
    """sfa_chunk_attend_paged, or with a mask sfa_tree_attend_paged."""
    dev = Q.get_device()
    n_q, h_q, dkq = Q.shape
    n_cells, h_kv, k_row = K.shape
    n_seq, dv = len_total.numel(), O.size(-1)
    _check_qkv(Q, K, V)
    code, o_code = _CODES.get(K.dtype), _CODES.get(O.dtype)
    q8 = code == SFA_Q8_0
    if code is None or k_row != (sfa_q8_0_row_bytes(dkq) if q8 else dkq):
        raise ValueError("Q and K must share a head size, K bf16, fp32 or q8_0 rows")
    if V is not None and V.shape != (n_cells, h_kv, sfa_q8_0_row_bytes(dv) if q8 else dv):
        raise ValueError("V must be [n_cells][h_kv][dv] like K")
    if O.shape != (n_q, h_q, dv) or o_code not in (SFA_F32, SFA_BF16):
        raise ValueError("O must be an fp32 or bf16 [n_q][h_q][dv] tensor")
    if lse is not None and (lse.shape != (n_q, h_q) or lse.dtype is not _F32):
        raise ValueError("lse must be an fp32 [n_q][h_q] tensor")
    for t in (Q, K, V, workspace):
        if t is not None and (t.get_device() != dev or not t.is_contiguous() or dev < 0):
            _no_tensor("every tensor", t, dev, "contiguous")
    for t in (O, lse):   # on the device, or in page-locked host memory
        if t is not None and (not t.is_contiguous() or t.get_device() != dev and (t.is_cuda or not t.is_pinned())):
            _no_tensor("an output", t, dev, "contiguous")
    table, cu = _int_rows("page_table", page_table, n_seq, dev), _ints("cu_new", cu_new, n_seq + 1, dev)
    total = _ints("len_total", len_total, n_seq, dev)
    tree = () if mask is None else (_int_rows("tree_mask", mask, n_q, dev), mask.size(1), part)
    ws_bytes = 0
    if workspace is None:
        sizes = (code, n_seq, n_q, h_q, h_kv, dkq, dv, V is not None, n_new_max, n_kv_max, o_code)
        ws_bytes = _chunk_workspace(dev, *sizes) if mask is None else _tree_workspace(dev, part, *sizes)
        if ws_bytes:
            workspace = _scratch(ws_bytes, dev, stream)
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    _call(lib().sfa_chunk_attend_paged if mask is None else lib().sfa_tree_attend_paged, dev, stream,
          Q.data_ptr(), K.data_ptr(),
          None if V is None else V.data_ptr(), code, n_cells, table, page_table.size(1), page_size,
          n_seq, n_q, h_q, h_kv, dkq, dv, scale, cu, total, *tree, n_new_max, n_kv_max, O.data_ptr(), o_code,
          None if lse is None else lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
          ws_bytes, None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


class _Rope(ctypes.Structure):
    """sfa_rope of include/sfa.h."""
    _fields_ = [("n_rot", ctypes.c_int32), ("pairs", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * (SFA_MAX_ROT // 2))]


class SfaRope:
    """A rotation by position for sfa_rotate_rows, made once: n_rot dims of a head turned in pairs, halves
    (j, j + n_rot/2) or, with pairs, adjacent dims (2j, 2j + 1), pair j by base ** (-2 j / n_rot) radians a
    position.  For contexts `factor` times the trained length: every frequency divided by it, or, given
    the trained length original_len, by parts (sfa_rope_frequencies); freqs gives any n_rot/2 others
    instead.  magnitude multiplies the turned dims.  freqs (a list of floats) holds what it turns by."""

    def __init__(self, n_rot: int, base: float = 10000.0, pairs: bool = False, factor: float = 1.0,
                 original_len: float = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 magnitude: float = 1.0, freqs=None):
        if n_rot < 2 or n_rot > SFA_MAX_ROT or n_rot % 2:
            raise ValueError(f"n_rot must be even, 2 to {SFA_MAX_ROT}")
        f = (ctypes.c_double * (n_rot // 2))()
        if freqs is None:
            _check("sfa_rope_frequencies", lib().sfa_rope_frequencies(n_rot, base, factor, original_len,
                                                                      beta_fast, beta_slow, f))
        else:
            freqs = [float(x) for x in freqs]
            if len(freqs) != n_rot // 2:
                raise ValueError(f"freqs must hold n_rot / 2 = {n_rot // 2} values")
            f[:] = freqs
        self._rope = _Rope()
        _check("sfa_rope_init", lib().sfa_rope_init(ctypes.addressof(self._rope), n_rot, int(bool(pairs)), f,
                                                    magnitude))
        self.n_rot, self.pairs, self.magnitude = n_rot, bool(pairs), float(self._rope.magnitude)
        self.freqs = list(f)


_ROTATION = struct.Struct("@QqqQqqiiiiii")     # sfa_row_rotation of include/sfa.h


def _rotation(src, dst, begin, n_rows, n_dst, to_cells, dev):
    """src [>= n_rows][d] or [..][h][d] into dst of the same heads, any strides but the last."""
    shape, to, st, dt = src.shape, dst.shape, src.stride(), dst.stride()
    code, out = _CODES.get(src.dtype, SFA_Q8_0), _CODES.get(dst.dtype, SFA_Q8_0)
    if len(shape) == 3:
        n, h, d = shape
        sh, dh = st[1], dt[1] if len(to) == 3 else 0
    else:
        n, d = shape if len(shape) == 2 else (-1, 0)
        h, sh, dh = 1, 0, 0
    if (h < 1 or d < 1 or n < n_rows or code == SFA_Q8_0 or src.get_device() != dev or (st[-1] != 1 and d > 1)):
        _no_tensor("rows to rotate", src, dev, f"bf16 or fp32, [>= {n_rows}][d] or [>= {n_rows}][h][d], each "
                   "head contiguous")
    if (to[1:] != shape[1:] or to[0] < n_dst or out == SFA_Q8_0 or dst.get_device() != dev
            or (dt[-1] != 1 and d > 1)):
        _no_tensor("rotated rows", dst, dev, f"bf16 or fp32, of their rows' heads, at least {n_dst} of them")
    return _ROTATION.pack(src.data_ptr(), st[0], sh, dst.data_ptr(), dt[0], dh, code, out, h, d, begin, to_cells)


def sfa_rotate_rows(rows, pos, rope: SfaRope, cells=(), slot=None, inverse: bool = False, dev_status=None,
                    stream=None):
    """Rows turned by their positions pos [n] int32 (negative: left out), in one launch: for every (x, out,
    begin) of rows, dims begin .. begin + n_rot of each head of x [n][d] or [n][h][d] into out (x itself:
    in place; views of any stride but the last's); for every (x, cache, begin) of cells, row i into row
    slot[i] of cache [n_cells][..].  fp32 rows may become bf16.  inverse turns the other way, which is
    also the way of gradients.  At most SFA_MAX_ROTATIONS of both."""
    rows, cells = list(rows), list(cells)
    if len(rows) + len(cells) > SFA_MAX_ROTATIONS:
        raise ValueError(f"at most {SFA_MAX_ROTATIONS} sets of rows per call")
    if cells and slot is None:
        raise ValueError("rows for cells need their slots")
    dev = _device_of(pos)
    n = pos.numel()
    at = _ints("pos", pos, n, dev)
    to = None if slot is None else _ints("slot", slot, n, dev)
    n_cells = cells[0][1].size(0) if cells else 0
    for _, cache, _ in cells:
        if cache.size(0) != n_cells:
            raise ValueError("caches of one call must have the same cells")
    packed = b"".join([_rotation(x, y, b, n, n, 0, dev) for x, y, b in rows]
                      + [_rotation(x, y, b, n, n_cells, 1, dev) for x, y, b in cells])
    if not packed:
        return
    _call(lib().sfa_rotate_rows, dev, stream, len(rows) + len(cells), packed, ctypes.addressof(rope._rope),
          int(bool(inverse)), at, n, to, n_cells,
          None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


def sfa_build_tree_maps(parent, cu_new, len_total, mask, q_pos, cached_pos=None, dev_status=None,
                        stream=None):
    """Drafted trees from their nodes' parents (parent [n] int32, indices within the node's own tree, -1:
    a root; the trees packed at cu_new [n_seq + 1], their ends at len_total): mask [n][words] int32 of
    the node itself and its ancestors, q_pos [n] (the cached tokens plus the node's depth) and, when
    given, cached_pos [n] (the last cached position).  Rows past the last node: 0 and -1."""
    dev = _device_of(parent)
    n, n_seq = parent.numel(), len_total.numel()
    rows = _int_rows("mask", mask, n, dev)
    _call(lib().sfa_build_tree_maps, dev, stream, _ints("parent", parent, n, dev),
          _ints("cu_new", cu_new, n_seq + 1, dev), _ints("len_total", len_total, n_seq, dev), n_seq, n, rows,
          mask.size(1), _ints("q_pos", q_pos, n, dev),
          None if cached_pos is None else _ints("cached_pos", cached_pos, n, dev),
          None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


def sfa_tree_accept(parent, token, target, cu_new, path, n_acc, next_token, root_target=None,
                    dev_status=None, stream=None):
    """The path of each tree that the model agrees with: from a root (the first one, or the one whose token
    is root_target [n_seq]) to the child whose token is target of its parent, and so on.  token, target
    [n]: the nodes' drafted tokens, the model's choice behind each.  path [n_seq][most] gets the nodes,
    then -1, n_acc [n_seq] their number, next_token [n_seq] the model's choice behind the last."""
    dev = _device_of(parent)
    n, n_seq = parent.numel(), n_acc.numel()
    rows = _int_rows("path", path, n_seq, dev)
    _call(lib().sfa_tree_accept, dev, stream, _ints("parent", parent, n, dev), _ints("token", token, n, dev),
          _ints("target", target, n, dev),
          None if root_target is None else _ints("root_target", root_target, n_seq, dev),
          _ints("cu_new", cu_new, n_seq + 1, dev), n_seq, n, rows, path.size(1),
          _ints("n_acc", n_acc, n_seq, dev), _ints("next_token", next_token, n_seq, dev),
          None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


_CELL_ROWS = struct.Struct("@Qq")     # sfa_cell_rows of include/sfa.h


def sfa_tree_commit(caches, slot, cu_new, path, n_acc, len_total, page_size: int, page_table, free_pages,
                    free_head, len_out, free_head_out, dev_status=None, stream=None):
    """The accepted nodes of each tree stay: in every cache ([n_cells][..], at most SFA_MAX_CELL_WRITES) the
    rows of path's first n_acc nodes move to the first cells of their step, len_out [n_seq] is where the
    sequences end then, and the pages behind go back to free_pages before entry free_head, which
    free_head_out replaces (either may be the tensor it follows from)."""
    caches = list(caches)
    if len(caches) > SFA_MAX_CELL_WRITES:
        raise ValueError(f"at most {SFA_MAX_CELL_WRITES} caches per call")
    dev = _device_of(slot)
    n, n_seq = slot.numel(), n_acc.numel()
    n_cells = caches[0].size(0) if caches else 0x7FFFFFFF
    packed = []
    for c in caches:
        if c.get_device() != dev or not c.is_contiguous() or c.size(0) != n_cells or c.dim() < 2:
            _no_tensor("a cache", c, dev, f"a contiguous [{n_cells}][..] tensor")
        packed.append(_CELL_ROWS.pack(c.data_ptr(), c.stride(0) * c.element_size()))
    rows = _int_rows("path", path, n_seq, dev)
    table = _int_rows("page_table", page_table, n_seq, dev)
    n_free = free_pages.numel()
    _call(lib().sfa_tree_commit, dev, stream, len(caches) if n_cells else 0, b"".join(packed), n_cells,
          _ints("slot", slot, n, dev), _ints("cu_new", cu_new, n_seq + 1, dev),
          _ints("len_total", len_total, n_seq, dev), n_seq, n, rows, path.size(1),
          _ints("n_acc", n_acc, n_seq, dev), page_size, table, page_table.size(1),
          _ints("free_pages", free_pages, n_free, dev), n_free, _ints("free_head", free_head, 1, dev),
          _ints("len_out", len_out, n_seq, dev), _ints("free_head_out", free_head_out, 1, dev),
          None if dev_status is None else _ints("dev_status", dev_status, 1, dev))


def sfa_read_device_status(dev_status, stream=None) -> int:
    out = ctypes.c_int32(0)
    rc = lib().sfa_read_device_status(_p(dev_status), ctypes.byref(out), _stream(stream))
    _check("sfa_read_device_status", rc)
    return int(out.value)
