"""Thin ctypes binding of ``libthdattn.so`` (see ``include/thd_attn.h``).

The ``thd_*`` functions here have the C names and argument order; they only
marshal arguments (torch tensors -> device pointers, the current torch stream
-> cudaStream_t) and return the C status code.  Every step of the
computation runs in the library's CUDA kernels; there is no Python or CPU
fallback: if the library is missing, ``lib()`` raises.

The lower-case helpers at the end (``attn_fwd``, ``attn_bwd``, ...) allocate
outputs, workspace and the device status word with torch and call the
``thd_*`` functions -- allocation and marshalling only.  With ``stream=`` (a
torch stream, or a cudaStream_t as an int) they allocate from that stream's
memory, where the kernels run, and keep what they were given and what they
return until both streams are done with it; ordering the two streams is the
caller's.  A raw handle's stream may end before the tensors do, so there the
caller also keeps the inputs until the work is done.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libthdattn.so")

THD_OK = 0
THD_ERR_INVALID_ARG = 1
THD_ERR_UNSUPPORTED = 2
THD_ERR_CUDA = 3
THD_ERR_TIMEOUT = 4
THD_ERR_WORKSPACE = 5
THD_DEV_ERR_NONZERO_START = 101
THD_DEV_ERR_NOT_MONOTONE = 102
THD_DEV_ERR_VALID_GT_PAD = 103
THD_DEV_ERR_NOT_DIVISIBLE = 104
THD_DEV_ERR_EXCEEDS_BUF = 105
THD_DEV_ERR_CAUSAL_LENGTHS = 106
THD_DEV_ERR_CAPACITY = 107
THD_DEV_ERR_DOC_ORDER = 108
THD_DEV_ERR_PAGE = 109
THD_DEV_ERR_KV_LEN = 110

THD_KERNEL_PLAN = 1
THD_KERNEL_FWD = 2
THD_KERNEL_BWD_PREP = 3
THD_KERNEL_BWD = 4
THD_KERNEL_BWD_DQ = 5
THD_KERNEL_LSE_MERGE = 6
THD_KERNEL_TAIL_ZERO = 7
THD_KERNEL_PARTITION = 8
THD_KERNEL_A2A = 9
THD_KERNEL_ROPE = 10
THD_KERNEL_DROPOUT = 11
THD_KERNEL_DOCS = 12
THD_KERNEL_BWD_JOIN = 13
THD_KERNEL_DECODE = 14
THD_KERNEL_DECODE_JOIN = 15
THD_KERNEL_CACHE_APPEND = 16
THD_KERNEL_CACHE_EVICT = 17
THD_KERNEL_DECODE_WEIGHTS = 18

THD_FWD_KERNEL_SINGLE = 1
THD_FWD_KERNEL_DUAL = 2

THD_CAUSAL_NONE = 0
THD_CAUSAL_TOP_LEFT = 1
THD_CAUSAL_BOTTOM_RIGHT = 2

THD_DTYPE_BF16 = 0
THD_DTYPE_FP32 = 1
THD_DTYPE_E4M3 = 2

THD_A2A_TO_GROUPS = 0
THD_A2A_TO_SHARDS = 1

_vp = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64
_f32 = ctypes.c_float
_f64 = ctypes.c_double
_sz = ctypes.c_size_t


class KvCache(ctypes.Structure):
    """thd_kv_cache.  The thd_* functions take one, or its bytes."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_exp", _vp), ("v_exp", _vp), ("block_table", _vp), ("kv_len", _vp),
                ("num_pages", _i64), ("table_stride", _i64), ("kv_stride", _i64 * 3), ("exp_stride", _i64 * 3),
                ("weight_stride", _i64 * 3), ("pos_stride", _i64 * 3), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


_pack_cache = struct.Struct("=6Q14q6i").pack   # the fields in order, without padding


def _c(cache):
    return cache if cache is None or isinstance(cache, bytes) else ctypes.byref(cache)


# name -> (restype, argtypes); mirrors include/thd_attn.h
SIGNATURES = {
    "thd_status_string": (ctypes.c_char_p, [_i32]),
    "thd_version": (_i32, []),
    "thd_workspace_size": (_sz, [_i32, _i64, _i64, _i32, _i32, _i32, _i32, _i32]),
    "thd_cp_partition": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "thd_attn_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32,
                            _i32, _f32, _i32, _i32, _vp, _sz, _vp, _vp]),
    "thd_attn_fwd_step": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32,
                                 _i32, _f32, _i32, _i32, _i32, _vp, _sz, _vp, _vp]),
    "thd_attn_fwd_step_bf16": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32,
                                      _i32, _i32, _f32, _i32, _i32, _i32, _vp, _sz, _vp, _vp]),
    "thd_attn_fwd_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32,
                                    _i32, _i32, _f32, _i32, _i32, _vp, _vp]),
    "thd_attn_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i32,
                            _i64, _i64, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _vp, _sz, _vp, _vp]),
    "thd_attn_score_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _i32, _i32,
                                  _i32, _f32, _i32, _i32, _f32, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "thd_attn_score_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i32,
                                  _i64, _i64, _i32, _i32, _i32, _i32, _f32, _i32, _i32, _f32, _vp, _vp, _vp, _vp,
                                  _vp, _sz, _vp, _vp]),
    "thd_score_workspace_size": (_sz, [_i32, _i64, _i64, _i32, _i32, _i32, _i32, _i32, _i32]),
    "thd_lse_merge": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _vp]),
    "thd_lse_merge_bf16": (_i32, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _vp]),
    "thd_grad_tail_zero": (_i32, [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _i32, _vp]),
    "thd_cp_a2a": (_i32, [_vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "thd_a2a_workspace_size": (_sz, [_i32, _i64, _i32, _i32, _i32, _i32, _i32, _i32]),
    "thd_attn_fwd_a2a": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _f32, _i32,
                                _i32, _vp, _sz, _vp, _vp]),
    "thd_attn_bwd_a2a": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                _i32, _f32, _i32, _i32, _vp, _sz, _vp, _vp]),
    "thd_rope": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp,
                        _vp, _i32, _i32, _i32, _vp]),
    "thd_dropout_add": (_i32, [_vp, _vp, _vp, _i64, _i64, _vp, _f64, _vp, _i32, _vp]),
    "thd_cache_append": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "thd_attn_decode": (_i32, [_vp, _vp, _i64, _vp, _vp, _i32, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp,
                               _vp]),
    "thd_decode_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i64, _i32]),
    "thd_cache_evict": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _sz, _vp, _vp]),
    "thd_evict_workspace_size": (_sz, [_i32, _i32, _i64, _i32]),
    "thd_profile_enable": (_i32, [_i32, _i32]),
    "thd_profile_read": (_i32, [_vp, _i32, _vp]),
    "thd_launch_count": (ctypes.c_uint64, []),
    "thd_test_arm_stall": (_i32, [_i32]),
    "thd_test_select_fwd_kernel": (_i32, [_i32]),
}

_LIB = None


def lib() -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m packed_sequence_context_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _p(x):
    """Device pointer of a tensor (or pass an int / None through)."""
    return x if x is None or isinstance(x, int) else x.data_ptr()


def _h(a):
    """Host address of a contiguous numpy array (or pass an int / None through)."""
    if a is None or isinstance(a, int):
        return a
    return a.ctypes.data


_RAW_STREAM = None
_HERE = contextlib.nullcontext()


def _s(stream):
    if stream is None:
        global _RAW_STREAM
        import torch
        if _RAW_STREAM is None:  # the handle without a Stream object around it (0.1 us instead of 3), where torch has it
            _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        return _RAW_STREAM(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ----------------------------------------------------------------- C names
def thd_status_string(status: int) -> str:
    return lib().thd_status_string(status).decode()


def thd_version() -> int:
    return lib().thd_version()


def thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, for_bwd) -> int:
    return lib().thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, for_bwd)


def thd_cp_partition(cu_seqlens, cu_seqlens_padded, B, cp_size, pad_between_seqs, cu_rank, cu_rank_padded,
                     cu_rank_half, token_map, token_map_capacity, dev_status, stream=None) -> int:
    return lib().thd_cp_partition(_p(cu_seqlens), _p(cu_seqlens_padded), B, cp_size, pad_between_seqs,
                                  _p(cu_rank), _p(cu_rank_padded), _p(cu_rank_half), _p(token_map),
                                  token_map_capacity, _p(dev_status), _s(stream))


def thd_attn_fwd(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, B, T_q,
                 T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size, pad_between_seqs, workspace, workspace_bytes,
                 dev_status, stream=None) -> int:
    return lib().thd_attn_fwd(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens_q), _p(cu_seqlens_kv),
                              _p(cu_seqlens_q_padded), _p(cu_seqlens_kv_padded), B, T_q, T_kv, Hq, Hkv, D, causal,
                              softmax_scale, cp_size, pad_between_seqs, _p(workspace), workspace_bytes,
                              _p(dev_status), _s(stream))


def thd_attn_fwd_step(q, k, v, o_part, lse_part, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded,
                      cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size,
                      pad_between_seqs, step, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_fwd_step(_p(q), _p(k), _p(v), _p(o_part), _p(lse_part), _p(cu_seqlens_q),
                                   _p(cu_seqlens_kv), _p(cu_seqlens_q_padded), _p(cu_seqlens_kv_padded), B, T_q,
                                   T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size, pad_between_seqs, step,
                                   _p(workspace), workspace_bytes, _p(dev_status), _s(stream))


def thd_attn_fwd_step_bf16(q, k, v, o_part, lse_part, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded,
                           cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size,
                           pad_between_seqs, step, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_fwd_step_bf16(_p(q), _p(k), _p(v), _p(o_part), _p(lse_part), _p(cu_seqlens_q),
                                        _p(cu_seqlens_kv), _p(cu_seqlens_q_padded), _p(cu_seqlens_kv_padded), B, T_q,
                                        T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size, pad_between_seqs, step,
                                        _p(workspace), workspace_bytes, _p(dev_status), _s(stream))


def thd_attn_fwd_noalloc(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded,
                         B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size, pad_between_seqs, dev_status,
                         stream=None) -> int:
    return lib().thd_attn_fwd_noalloc(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens_q), _p(cu_seqlens_kv),
                                      _p(cu_seqlens_q_padded), _p(cu_seqlens_kv_padded), B, T_q, T_kv, Hq, Hkv, D,
                                      causal, softmax_scale, cp_size, pad_between_seqs, _p(dev_status), _s(stream))


def thd_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, dq_rows, dkv_rows, cu_seqlens_q, cu_seqlens_kv,
                 cu_seqlens_q_padded, cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale,
                 cp_size, pad_between_seqs, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_bwd(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(dout), _p(dq), _p(dk), _p(dv), dq_rows,
                              dkv_rows, _p(cu_seqlens_q), _p(cu_seqlens_kv), _p(cu_seqlens_q_padded),
                              _p(cu_seqlens_kv_padded), B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size,
                              pad_between_seqs, _p(workspace), workspace_bytes, _p(dev_status), _s(stream))


def thd_attn_score_fwd(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, B,
                       T_q, T_kv, Hq, Hkv, D, causal, softmax_scale, cp_size, pad_between_seqs, softcap, dist_slopes,
                       doc_q, doc_kv, prefix_len, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_score_fwd(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens_q), _p(cu_seqlens_kv),
                                    _p(cu_seqlens_q_padded), _p(cu_seqlens_kv_padded), B, T_q, T_kv, Hq, Hkv, D,
                                    causal, softmax_scale, cp_size, pad_between_seqs, softcap, _p(dist_slopes),
                                    _p(doc_q), _p(doc_kv), _p(prefix_len), _p(workspace), workspace_bytes,
                                    _p(dev_status), _s(stream))


def thd_attn_score_bwd(q, k, v, o, lse, dout, dq, dk, dv, dq_rows, dkv_rows, cu_seqlens_q, cu_seqlens_kv,
                       cu_seqlens_q_padded, cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale,
                       cp_size, pad_between_seqs, softcap, dist_slopes, doc_q, doc_kv, prefix_len, workspace,
                       workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_score_bwd(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(dout), _p(dq), _p(dk), _p(dv), dq_rows,
                                    dkv_rows, _p(cu_seqlens_q), _p(cu_seqlens_kv), _p(cu_seqlens_q_padded),
                                    _p(cu_seqlens_kv_padded), B, T_q, T_kv, Hq, Hkv, D, causal, softmax_scale,
                                    cp_size, pad_between_seqs, softcap, _p(dist_slopes), _p(doc_q), _p(doc_kv),
                                    _p(prefix_len), _p(workspace), workspace_bytes, _p(dev_status), _s(stream))


def thd_score_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, has_docs, for_bwd) -> int:
    return lib().thd_score_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, has_docs, for_bwd)


def thd_lse_merge(o_acc, lse_acc, o_part, lse_part, T, H, D, stream=None) -> int:
    return lib().thd_lse_merge(_p(o_acc), _p(lse_acc), _p(o_part), _p(lse_part), T, H, D, _s(stream))


def thd_lse_merge_bf16(o_acc, lse_acc, o_part, lse_part, T, H, D, stream=None) -> int:
    return lib().thd_lse_merge_bf16(_p(o_acc), _p(lse_acc), _p(o_part), _p(lse_part), T, H, D, _s(stream))


def thd_grad_tail_zero(dq, dk, dv, dq_rows, dkv_rows, Hq, Hkv, D, cu_seqlens_q_padded, cu_seqlens_kv_padded, B,
                       host_knows_no_tail, stream=None) -> int:
    return lib().thd_grad_tail_zero(_p(dq), _p(dk), _p(dv), dq_rows, dkv_rows, Hq, Hkv, D, _p(cu_seqlens_q_padded),
                                    _p(cu_seqlens_kv_padded), B, host_knows_no_tail, _s(stream))


def thd_cp_a2a(src, dst, cu_seqlens_padded, B, T, H, D, cp_size, a2a_size, direction, dev_status,
               stream=None) -> int:
    return lib().thd_cp_a2a(_p(src), _p(dst), _p(cu_seqlens_padded), B, T, H, D, cp_size, a2a_size, direction,
                            _p(dev_status), _s(stream))


def thd_a2a_workspace_size(B, T, Hq, Hkv, D, cp_size, a2a_size, for_bwd) -> int:
    return lib().thd_a2a_workspace_size(B, T, Hq, Hkv, D, cp_size, a2a_size, for_bwd)


def thd_attn_fwd_a2a(q, k, v, o, lse, cu_seqlens, cu_seqlens_padded, B, T, Hq, Hkv, D, causal, softmax_scale,
                     cp_size, a2a_size, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_fwd_a2a(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu_seqlens), _p(cu_seqlens_padded), B, T,
                                  Hq, Hkv, D, causal, softmax_scale, cp_size, a2a_size, _p(workspace),
                                  workspace_bytes, _p(dev_status), _s(stream))


def thd_attn_bwd_a2a(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens, cu_seqlens_padded, B, T, Hq, Hkv, D, causal,
                     softmax_scale, cp_size, a2a_size, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_bwd_a2a(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(dout), _p(dq), _p(dk), _p(dv),
                                  _p(cu_seqlens), _p(cu_seqlens_padded), B, T, Hq, Hkv, D, causal, softmax_scale,
                                  cp_size, a2a_size, _p(workspace), workspace_bytes, _p(dev_status), _s(stream))


def thd_rope(q_in, k_in, q_out, k_out, q_in_stride, k_in_stride, q_out_stride, k_out_stride, T, Hq, Hkv, D, rot_dim,
             positions, n_axes, inv_freq, axis_of, adjacent, inverse, dtype, stream=None) -> int:
    return lib().thd_rope(_p(q_in), _p(k_in), _p(q_out), _p(k_out), q_in_stride, k_in_stride, q_out_stride,
                          k_out_stride, T, Hq, Hkv, D, rot_dim, _p(positions), n_axes, _h(inv_freq), _h(axis_of),
                          adjacent, inverse, dtype, _s(stream))


def thd_dropout_add(x, residual, out, T, C, row_ids, p, rng, dtype, stream=None) -> int:
    return lib().thd_dropout_add(_p(x), _p(residual), _p(out), T, C, _p(row_ids), p, _p(rng), dtype, _s(stream))


def thd_cache_append(cache, k, v, k_stride, v_stride, T, cu_seqlens, weight, pos, tokens_seen, dev_status,
                     stream=None) -> int:
    return lib().thd_cache_append(_c(cache), _p(k), _p(v), k_stride, v_stride, T, _p(cu_seqlens),
                                  _p(weight), _p(pos), _p(tokens_seen), _p(dev_status), _s(stream))


def thd_attn_decode(cache, q, q_stride, o, lse, Hq, softmax_scale, softcap, dist_slopes, kv_start, pos, tokens_seen,
                    weight_in, weight_out, workspace, workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_attn_decode(_c(cache), _p(q), q_stride, _p(o), _p(lse), Hq, softmax_scale, softcap, _p(dist_slopes),
                                 _p(kv_start), _p(pos), _p(tokens_seen), _p(weight_in), _p(weight_out), _p(workspace),
                                 workspace_bytes, _p(dev_status), _s(stream))


def thd_decode_workspace_size(B, Hq, Hkv, D, capacity, has_weights) -> int:
    return lib().thd_decode_workspace_size(B, Hq, Hkv, D, capacity, has_weights)


def thd_cache_evict(cache, weight_in, weight_out, pos_in, pos_out, tokens_seen, budget, sinks, recent, new_len, workspace,
                    workspace_bytes, dev_status, stream=None) -> int:
    return lib().thd_cache_evict(_c(cache), _p(weight_in), _p(weight_out), _p(pos_in), _p(pos_out), _p(tokens_seen), budget,
                                 sinks, recent, _p(new_len), _p(workspace), workspace_bytes, _p(dev_status), _s(stream))


def thd_evict_workspace_size(B, Hkv, capacity, budget) -> int:
    return lib().thd_evict_workspace_size(B, Hkv, capacity, budget)


def thd_profile_enable(kernel_id: int, max_records: int) -> int:
    return lib().thd_profile_enable(kernel_id, max_records)


def thd_profile_read(max_out: int = 4096) -> list[float]:
    buf = (ctypes.c_float * max_out)()
    n = ctypes.c_int(0)
    rc = lib().thd_profile_read(ctypes.cast(buf, _vp), max_out, ctypes.cast(ctypes.pointer(n), _vp))
    if rc != THD_OK:
        raise RuntimeError(f"thd_profile_read: {thd_status_string(rc)}")
    return [buf[i] for i in range(n.value)]


def thd_launch_count() -> int:
    return lib().thd_launch_count()


def thd_test_arm_stall(kernel_id: int) -> int:
    return lib().thd_test_arm_stall(kernel_id)


def thd_test_select_fwd_kernel(which: int) -> int:
    return lib().thd_test_select_fwd_kernel(which)


# ----------------------------------------------------------------- helpers
class ThdError(RuntimeError):
    def __init__(self, where: str, code: int):
        super().__init__(f"{where}: {thd_status_string(code)} ({code})")
        self.code = code


def _check(where: str, rc: int):
    if rc != THD_OK:
        raise ThdError(where, rc)


def check_status(dev_status) -> int:
    """Synchronise and raise on a nonzero device status word."""
    code = int(dev_status.item())
    if code != 0:
        raise ThdError("device", code)
    return code


def _need(where: str, ok: bool):
    """Refuse a call whose tensors the library could not tell from right ones
    (it sees pointers): wrong type, shape, device or layout."""
    if not ok:
        raise ThdError(where, THD_ERR_INVALID_ARG)


def _dtype(where: str, t) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return THD_DTYPE_BF16
    if t.dtype is torch.float32:
        return THD_DTYPE_FP32
    raise ThdError(where, THD_ERR_UNSUPPORTED)


def _current(where: str, t) -> int:
    """The tensor's device index; it must be the current CUDA device, where
    the library launches."""
    import torch
    dev = t.get_device()  # -1 on the CPU
    _need(where, dev >= 0 and dev == torch.cuda.current_device())
    return dev


def _aside(stream):
    """The torch stream of a call that does not run on the current one, else
    None.  0 and 1 are the legacy default stream."""
    if stream is None:
        return None
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.default_stream() if handle in (0, 1) else torch.cuda.ExternalStream(handle)
    return None if stream == torch.cuda.current_stream() else stream


def _alloc_on(side):
    """Where the buffers of a call are made: a block of the current stream's
    memory would be free for the current stream's next tensor once the helper
    drops it, and may still be in use by what that stream ran before."""
    if side is None:
        return _HERE
    import torch
    return torch.cuda.stream(side)


def _keep(side, stream, given, made):
    """After a launch on another stream: the memory of what the call was given
    (unless by a raw handle) and of what it returns stays until both streams
    are done with it."""
    if side is None:
        return
    import torch
    cur = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        for t in given:
            if isinstance(t, torch.Tensor):
                t.record_stream(side)
    for t in made:
        if t is not None and not any(t is g for g in given):
            t.record_stream(cur)


def _workspace(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def attn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded=None, cu_seqlens_kv_padded=None, *,
             cp_size=1, causal=True, softmax_scale=None, pad_between_seqs=-1, out=None, lse=None,
             dev_status=None, workspace=None, stream=None):
    """Allocate O [T_q,Hq,D] bf16, lse [Hq,T_q] fp32 and call thd_attn_fwd.
    Returns (o, lse, dev_status); read dev_status after synchronising."""
    import torch
    T_q, Hq, D = q.shape
    T_kv, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    side = _aside(stream)
    with _alloc_on(side):
        o = torch.empty_like(q) if out is None else out
        l = torch.empty((Hq, T_q), dtype=torch.float32, device=q.device) if lse is None else lse
        st = torch.zeros(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        nbytes = thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, 0)
        ws = _workspace(nbytes, q.device) if workspace is None else workspace
    _check("thd_attn_fwd", thd_attn_fwd(q, k, v, o, l, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded,
                                        cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, int(causal), scale,
                                        cp_size, pad_between_seqs, ws, ws.numel(), st, stream))
    _keep(side, stream, (q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, out, lse,
                         dev_status, workspace), (o, l, st))
    return o, l, st


def attn_fwd_step(q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded=None, cu_seqlens_kv_padded=None, *,
                  step, cp_size=1, causal=True, softmax_scale=None, pad_between_seqs=-1, out=None, lse=None,
                  stream=None):
    """One ring step's materialised partial: (o_part fp32 [T_q,Hq,D], lse_part [Hq,T_q], dev_status)."""
    import torch
    T_q, Hq, D = q.shape
    T_kv, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    side = _aside(stream)
    with _alloc_on(side):
        o = torch.empty((T_q, Hq, D), dtype=torch.float32, device=q.device) if out is None else out
        l = torch.empty((Hq, T_q), dtype=torch.float32, device=q.device) if lse is None else lse
        st = torch.zeros(1, dtype=torch.int32, device=q.device)
        ws = _workspace(thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, 0), q.device)
    _check("thd_attn_fwd_step", thd_attn_fwd_step(q, k, v, o, l, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded,
                                                  cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, int(causal),
                                                  scale, cp_size, pad_between_seqs, step, ws, ws.numel(), st,
                                                  stream))
    _keep(side, stream, (q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, out, lse),
          (o, l, st))
    return o, l, st


def attn_fwd_step_bf16(q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded=None, cu_seqlens_kv_padded=None,
                       *, step, cp_size=1, causal=True, softmax_scale=None, pad_between_seqs=-1, out=None, lse=None,
                       dev_status=None, workspace=None, stream=None):
    """One ring step's partial in bf16: (o_part bf16 [T_q,Hq,D], lse_part fp32 [Hq,T_q], dev_status)."""
    import torch
    T_q, Hq, D = q.shape
    T_kv, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    side = _aside(stream)
    with _alloc_on(side):
        o = torch.empty((T_q, Hq, D), dtype=torch.bfloat16, device=q.device) if out is None else out
        l = torch.empty((Hq, T_q), dtype=torch.float32, device=q.device) if lse is None else lse
        st = torch.zeros(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        ws = _workspace(thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, 0), q.device) if workspace is None \
            else workspace
    _check("thd_attn_fwd_step_bf16", thd_attn_fwd_step_bf16(q, k, v, o, l, cu_seqlens_q, cu_seqlens_kv,
                                                            cu_seqlens_q_padded, cu_seqlens_kv_padded, B, T_q, T_kv,
                                                            Hq, Hkv, D, int(causal), scale, cp_size,
                                                            pad_between_seqs, step, ws, ws.numel(), st, stream))
    _keep(side, stream, (q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, out, lse,
                         dev_status, workspace), (o, l, st))
    return o, l, st


def attn_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded=None,
             cu_seqlens_kv_padded=None, *, cp_size=1, causal=True, softmax_scale=None, pad_between_seqs=-1,
             dq_rows=None, dkv_rows=None, dq=None, dk=None, dv=None, dev_status=None, workspace=None, stream=None):
    """Allocate dQ/dK/dV (with optional slack rows) and call thd_attn_bwd.
    Returns (dq, dk, dv, dev_status)."""
    import torch
    T_q, Hq, D = q.shape
    T_kv, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    dq_rows = T_q if dq_rows is None else dq_rows
    dkv_rows = T_kv if dkv_rows is None else dkv_rows
    given = (q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, dq, dk, dv,
             dev_status, workspace)
    side = _aside(stream)
    with _alloc_on(side):
        dq = torch.empty((dq_rows, Hq, D), dtype=q.dtype, device=q.device) if dq is None else dq
        dk = torch.empty((dkv_rows, Hkv, D), dtype=q.dtype, device=q.device) if dk is None else dk
        dv = torch.empty((dkv_rows, Hkv, D), dtype=q.dtype, device=q.device) if dv is None else dv
        st = torch.zeros(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        nbytes = thd_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size, 1)
        ws = _workspace(nbytes, q.device) if workspace is None else workspace
    _check("thd_attn_bwd", thd_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, dq_rows, dkv_rows, cu_seqlens_q,
                                        cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, B, T_q, T_kv, Hq,
                                        Hkv, D, int(causal), scale, cp_size, pad_between_seqs, ws, ws.numel(), st,
                                        stream))
    _keep(side, stream, given, (dq, dk, dv, st))
    return dq, dk, dv, st


def _score_checks(w, q, k, v, more, offsets, dist_slopes, doc_q, doc_kv, prefix_len, workspace):
    """What the library cannot see of a scored call: types, shapes, layout and
    device of its tensors.  `more`: (tensor, shape, dtype) triples."""
    import torch
    dev = _current(w, q)
    _need(w, workspace is None or workspace.get_device() == dev and workspace.is_contiguous())
    qs, ks = q.shape, k.shape
    B = offsets[0].numel() - 1
    bf16, i32 = torch.bfloat16, torch.int32
    triples = [(q, qs, bf16), (k, (ks[0], ks[1], qs[2]), bf16), (v, ks, bf16), *more]
    for t in offsets:
        if t is not None:
            triples.append((t, (B + 1,), i32))
    if dist_slopes is not None:
        triples.append((dist_slopes, (qs[1],), torch.float32))
    if doc_q is not None:
        triples.append((doc_q, (qs[0],), i32))
    if doc_kv is not None:
        triples.append((doc_kv, (ks[0],), i32))
    if prefix_len is not None:
        triples.append((prefix_len, (B,), i32))
    for t, shape, dtype in triples:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                                  and t.is_contiguous()):
            _need(w, False)
    return B, qs[0], ks[0], qs[1], ks[1], qs[2]


def attn_score_fwd(q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded=None, cu_seqlens_kv_padded=None, *,
                   softcap=0.0, dist_slopes=None, doc_q=None, doc_kv=None, prefix_len=None, cp_size=1, causal=True,
                   softmax_scale=None, pad_between_seqs=-1, out=None, lse=None, dev_status=None, workspace=None,
                   stream=None):
    """attn_fwd with capped scores (softcap), a bias by distance (dist_slopes
    fp32 [Hq]), documents (doc_q int32 [T_q], doc_kv [T_kv]) and prefixes
    (prefix_len int32 [B]).  Returns (o, lse, dev_status)."""
    import torch
    w = "thd_attn_score_fwd"
    _need(w, q.dim() == 3 and k.dim() == 3)
    more = [] if out is None and lse is None and dev_status is None else \
        [(out, q.shape, torch.bfloat16), (lse, (q.shape[1], q.shape[0]), torch.float32), (dev_status, (1,), torch.int32)]
    B, T_q, T_kv, Hq, Hkv, D = _score_checks(
        w, q, k, v, more, (cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded), dist_slopes,
        doc_q, doc_kv, prefix_len, workspace)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    side = _aside(stream)
    with _alloc_on(side):
        o = torch.empty_like(q) if out is None else out
        l = torch.empty((Hq, T_q), dtype=torch.float32, device=q.device) if lse is None else lse
        st = torch.empty(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        if workspace is None:
            workspace = _workspace(thd_score_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size,
                                                            int(doc_q is not None), 0), q.device)
    _check(w, thd_attn_score_fwd(q, k, v, o, l, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded,
                                 cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, int(causal), scale, cp_size,
                                 pad_between_seqs, softcap, dist_slopes, doc_q, doc_kv, prefix_len, workspace,
                                 workspace.numel(), st, stream))
    _keep(side, stream, (q, k, v, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, dist_slopes,
                         doc_q, doc_kv, prefix_len, out, lse, dev_status, workspace), (o, l, st))
    return o, l, st


def attn_score_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded=None,
                   cu_seqlens_kv_padded=None, *, softcap=0.0, dist_slopes=None, doc_q=None, doc_kv=None,
                   prefix_len=None, cp_size=1, causal=True, softmax_scale=None, pad_between_seqs=-1, dq_rows=None,
                   dkv_rows=None, dq=None, dk=None, dv=None, dev_status=None, workspace=None, stream=None):
    """Gradients of attn_score_fwd (same modifications), with optional slack
    rows as in attn_bwd.  Returns (dq, dk, dv, dev_status)."""
    import torch
    w = "thd_attn_score_bwd"
    _need(w, q.dim() == 3 and k.dim() == 3)
    bf16 = torch.bfloat16
    dq_rows = q.shape[0] if dq_rows is None else dq_rows
    dkv_rows = k.shape[0] if dkv_rows is None else dkv_rows
    qs, ks = (dq_rows, *q.shape[1:]), (dkv_rows, *k.shape[1:])
    more = [(o, q.shape, bf16), (dout, q.shape, bf16), (lse, (q.shape[1], q.shape[0]), torch.float32),
            (dq, qs, bf16), (dk, ks, bf16), (dv, ks, bf16), (dev_status, (1,), torch.int32)]
    B, T_q, T_kv, Hq, Hkv, D = _score_checks(
        w, q, k, v, more, (cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded), dist_slopes,
        doc_q, doc_kv, prefix_len, workspace)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    given = (q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_kv, cu_seqlens_q_padded, cu_seqlens_kv_padded, dist_slopes,
             doc_q, doc_kv, prefix_len, dq, dk, dv, dev_status, workspace)
    side = _aside(stream)
    with _alloc_on(side):
        dq = torch.empty(qs, dtype=bf16, device=q.device) if dq is None else dq
        dk = torch.empty(ks, dtype=bf16, device=q.device) if dk is None else dk
        dv = torch.empty(ks, dtype=bf16, device=q.device) if dv is None else dv
        st = torch.empty(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        if workspace is None:
            workspace = _workspace(thd_score_workspace_size(B, T_q, T_kv, Hq, Hkv, D, cp_size,
                                                            int(doc_q is not None), 1), q.device)
    _check(w, thd_attn_score_bwd(q, k, v, o, lse, dout, dq, dk, dv, dq_rows, dkv_rows, cu_seqlens_q, cu_seqlens_kv,
                                 cu_seqlens_q_padded, cu_seqlens_kv_padded, B, T_q, T_kv, Hq, Hkv, D, int(causal),
                                 scale, cp_size, pad_between_seqs, softcap, dist_slopes, doc_q, doc_kv, prefix_len,
                                 workspace, workspace.numel(), st, stream))
    _keep(side, stream, given, (dq, dk, dv, st))
    return dq, dk, dv, st


def cp_partition(cu_seqlens, cu_seqlens_padded=None, *, cp_size, pad_between_seqs=-1, token_map_capacity=None,
                 stream=None):
    """Per-rank partition via thd_cp_partition.  Returns a dict of device
    int32 tensors (cu_rank [cp,B+1], cu_rank_padded [cp,B+1], cu_rank_half
    [cp,2,B+1], token_map [capacity]) and the status word."""
    import torch
    B = cu_seqlens.numel() - 1
    dev = cu_seqlens.device
    cap = int(token_map_capacity) if token_map_capacity is not None else 0
    side = _aside(stream)
    with _alloc_on(side):
        out = {
            "cu_rank": torch.empty((cp_size, B + 1), dtype=torch.int32, device=dev),
            "cu_rank_padded": torch.empty((cp_size, B + 1), dtype=torch.int32, device=dev),
            "cu_rank_half": torch.empty((cp_size, 2, B + 1), dtype=torch.int32, device=dev),
            "token_map": torch.empty(max(cap, 1), dtype=torch.int32, device=dev),
        }
        st = torch.zeros(1, dtype=torch.int32, device=dev)
    _check("thd_cp_partition", thd_cp_partition(cu_seqlens, cu_seqlens_padded, B, cp_size, pad_between_seqs,
                                                out["cu_rank"], out["cu_rank_padded"], out["cu_rank_half"],
                                                out["token_map"] if cap else None, cap, st, stream))
    _keep(side, stream, (cu_seqlens, cu_seqlens_padded), (*out.values(), st))
    return out, st


def lse_merge(o_acc, lse_acc, o_part, lse_part, stream=None):
    """In-place merge of (o_part, lse_part) into (o_acc, lse_acc)."""
    T, H, D = o_acc.shape
    _check("thd_lse_merge", thd_lse_merge(o_acc, lse_acc, o_part, lse_part, T, H, D, stream))
    _keep(_aside(stream), stream, (o_acc, lse_acc, o_part, lse_part), ())


def lse_merge_bf16(o_acc, lse_acc, o_part, lse_part, stream=None):
    """In-place merge of a bf16 partial (o_part, lse_part) into the fp32 (o_acc, lse_acc)."""
    T, H, D = o_acc.shape
    _check("thd_lse_merge_bf16", thd_lse_merge_bf16(o_acc, lse_acc, o_part, lse_part, T, H, D, stream))
    _keep(_aside(stream), stream, (o_acc, lse_acc, o_part, lse_part), ())


def grad_tail_zero(dq, dk, dv, cu_seqlens_q_padded, cu_seqlens_kv_padded, host_knows_no_tail=False, stream=None):
    Hq, D = dq.shape[1], dq.shape[2]
    Hkv = dk.shape[1]
    B = cu_seqlens_q_padded.numel() - 1
    _check("thd_grad_tail_zero", thd_grad_tail_zero(dq, dk, dv, dq.shape[0], dk.shape[0], Hq, Hkv, D,
                                                    cu_seqlens_q_padded, cu_seqlens_kv_padded, B,
                                                    int(host_knows_no_tail), stream))
    _keep(_aside(stream), stream, (dq, dk, dv, cu_seqlens_q_padded, cu_seqlens_kv_padded), ())


def cp_a2a(src, cu_seqlens_padded, *, cp_size, a2a_size, direction, out=None, dev_status=None, stream=None):
    """Allocate the other layout and call thd_cp_a2a.  THD_A2A_TO_GROUPS:
    src shards [cp, T/cp, H, D] -> [a2a, T, H/a2a, D]; THD_A2A_TO_SHARDS: the
    reverse.  Returns (dst, dev_status)."""
    import torch
    if direction == THD_A2A_TO_GROUPS:
        cp, rows_r, H, D = src.shape
        T = cp * rows_r
        shape = (a2a_size, T, H // a2a_size, D)
    else:
        a, T, Hg, D = src.shape
        H = a * Hg
        shape = (cp_size, T // cp_size, H, D)
    B = cu_seqlens_padded.numel() - 1
    side = _aside(stream)
    with _alloc_on(side):
        dst = torch.empty(shape, dtype=src.dtype, device=src.device) if out is None else out
        st = torch.zeros(1, dtype=torch.int32, device=src.device) if dev_status is None else dev_status
    _check("thd_cp_a2a", thd_cp_a2a(src, dst, cu_seqlens_padded, B, T, H, D, cp_size, a2a_size, direction, st,
                                    stream))
    _keep(side, stream, (src, cu_seqlens_padded, out, dev_status), (dst, st))
    return dst, st


def attn_fwd_a2a(q, k, v, cu_seqlens, cu_seqlens_padded, *, cp_size, a2a_size, causal=True, softmax_scale=None,
                 out=None, lse=None, dev_status=None, workspace=None, stream=None):
    """Attention through the emulated A2A / hierarchical layer on shards
    q [cp, T/cp, Hq, D], k, v [cp, T/cp, Hkv, D].  Returns (o shards,
    lse [Hq, T] in global row order, dev_status)."""
    import torch
    cp, rows_r, Hq, D = q.shape
    Hkv = k.shape[2]
    T = cp * rows_r
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    side = _aside(stream)
    with _alloc_on(side):
        o = torch.empty_like(q) if out is None else out
        l = torch.empty((Hq, T), dtype=torch.float32, device=q.device) if lse is None else lse
        st = torch.zeros(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        nbytes = thd_a2a_workspace_size(B, T, Hq, Hkv, D, cp_size, a2a_size, 0)
        ws = _workspace(nbytes, q.device) if workspace is None else workspace
    _check("thd_attn_fwd_a2a", thd_attn_fwd_a2a(q, k, v, o, l, cu_seqlens, cu_seqlens_padded, B, T, Hq, Hkv, D,
                                                int(causal), scale, cp_size, a2a_size, ws, ws.numel(), st, stream))
    _keep(side, stream, (q, k, v, cu_seqlens, cu_seqlens_padded, out, lse, dev_status, workspace), (o, l, st))
    return o, l, st


def attn_bwd_a2a(q, k, v, o, lse, dout, cu_seqlens, cu_seqlens_padded, *, cp_size, a2a_size, causal=True,
                 softmax_scale=None, dq=None, dk=None, dv=None, dev_status=None, workspace=None, stream=None):
    """Gradients through the emulated A2A / hierarchical layer; shards in and
    out.  Returns (dq, dk, dv, dev_status)."""
    import torch
    cp, rows_r, Hq, D = q.shape
    Hkv = k.shape[2]
    T = cp * rows_r
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    given = (q, k, v, o, lse, dout, cu_seqlens, cu_seqlens_padded, dq, dk, dv, dev_status, workspace)
    side = _aside(stream)
    with _alloc_on(side):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        st = torch.zeros(1, dtype=torch.int32, device=q.device) if dev_status is None else dev_status
        nbytes = thd_a2a_workspace_size(B, T, Hq, Hkv, D, cp_size, a2a_size, 1)
        ws = _workspace(nbytes, q.device) if workspace is None else workspace
    _check("thd_attn_bwd_a2a", thd_attn_bwd_a2a(q, k, v, o, lse, dout, dq, dk, dv, cu_seqlens, cu_seqlens_padded, B,
                                                T, Hq, Hkv, D, int(causal), scale, cp_size, a2a_size, ws, ws.numel(),
                                                st, stream))
    _keep(side, stream, given, (dq, dk, dv, st))
    return dq, dk, dv, st


def _rope_rows(where, like, t, T, H, D):
    """The stride, in elements, of rows of [H, D] whose heads are contiguous.
    A dimension of size 1 may carry any stride."""
    _need(where, t.shape == (T, H, D) and t.dtype is like.dtype and t.get_device() == like.get_device())
    s0, s1, s2 = t.stride()
    _need(where, (s2 == 1 or D == 1) and (s1 == D or H == 1))
    return s0 if T > 1 else max(s0, H * D)


def rope(q, k, positions, inv_freq, axis_of=None, *, adjacent=False, inverse=False, q_out=None, k_out=None,
         stream=None):
    """Rotary positions on q [T, Hq, D] and k [T, Hkv, D] (k may be None).
    positions int32 [n_axes, T] (or [T]); inv_freq numpy float64
    [rot_dim / 2] and axis_of numpy uint8 [rot_dim / 2] on the host (None: all
    axis 0).  q and k may be slices of a fused projection (heads contiguous,
    any row stride); outputs are new contiguous tensors unless given (q_out=q:
    in place).  inverse=True: the gradients of the inputs.  Returns (q_out,
    k_out)."""
    import numpy as np
    import torch
    w = "thd_rope"
    _need(w, q.dim() == 3 and (k is None or k.dim() == 3) and positions.dim() in (1, 2))
    T, Hq, D = q.shape
    dev = _current(w, q)
    dt = _dtype(w, q)
    inv = np.ascontiguousarray(inv_freq, dtype=np.float64)
    n_axes = positions.shape[0] if positions.dim() == 2 else 1
    axis = np.zeros(inv.size, np.uint8) if axis_of is None else np.ascontiguousarray(axis_of)
    if axis.dtype != np.uint8:  # numbers that a byte would change into others
        _need(w, axis.dtype.kind in "iufb" and axis.size > 0 and 0 <= axis.min() and axis.max() < n_axes)
        byte = axis.astype(np.uint8)
        _need(w, np.array_equal(byte, axis))
        axis = byte
    _need(w, inv.ndim == 1 and axis.shape == inv.shape and positions.dtype is torch.int32 and
          positions.shape[-1] == T and positions.get_device() == dev and positions.is_contiguous())
    given = (q, k, positions, q_out, k_out)
    s_q, s_qo = _rope_rows(w, q, q, T, Hq, D), Hq * D
    if q_out is not None:
        s_qo = _rope_rows(w, q, q_out, T, Hq, D)
    Hkv = s_k = s_ko = 0
    if k is not None:
        Hkv = k.shape[1]
        s_k, s_ko = _rope_rows(w, q, k, T, Hkv, D), Hkv * D
        if k_out is not None:
            s_ko = _rope_rows(w, q, k_out, T, Hkv, D)
    else:
        _need(w, k_out is None)
    side = _aside(stream)
    with _alloc_on(side):
        if q_out is None:
            q_out = q.new_empty((T, Hq, D))
        if k is not None and k_out is None:
            k_out = k.new_empty((T, Hkv, D))
    _check(w, thd_rope(q, k, q_out, k_out, s_q, s_k, s_qo, s_ko, T, Hq, Hkv, D, 2 * inv.size, positions, n_axes, inv,
                       axis, int(adjacent), int(inverse), dt, stream))
    _keep(side, stream, given, (q_out, k_out))
    return q_out, k_out


def dropout_add(x, rng, p, *, residual=None, row_ids=None, out=None, stream=None):
    """residual + dropout(x) on contiguous rows [..., C] (the rows are the
    flattened leading dimensions), the mask drawn from rng (device int64 or
    uint64 [2]: seed, offset) and each row's number (row_ids int32 [rows], or
    its index).  On the output's gradient without a residual: the gradient of
    x.  out may be x or residual.  Returns out."""
    import torch
    w = "thd_dropout_add"
    dev = _current(w, x)
    dt = _dtype(w, x)
    _need(w, x.dim() >= 1)
    shape, dtype = x.shape, x.dtype
    C = shape[-1]
    T = x.numel() // C if C else 0
    given = (x, rng, residual, row_ids, out)
    if out is not None:
        _need(w, out.shape == shape and out.dtype is dtype and out.get_device() == dev and out.is_contiguous())
    if residual is not None:
        _need(w, residual.shape == shape and residual.dtype is dtype and residual.get_device() == dev and
              residual.is_contiguous())
    if row_ids is not None:
        _need(w, row_ids.dtype is torch.int32 and row_ids.numel() == T and row_ids.get_device() == dev and
              row_ids.is_contiguous())
    _need(w, x.is_contiguous() and rng.get_device() == dev and rng.numel() == 2 and rng.is_contiguous() and
          (rng.dtype is torch.int64 or rng.dtype is torch.uint64))
    side = _aside(stream)
    if out is None:
        with _alloc_on(side):
            out = torch.empty_like(x)
    _check(w, thd_dropout_add(x, residual, out, T, C, row_ids, p, rng, dt, stream))
    _keep(side, stream, given, (out,))
    return out


def _row_stride(where, like, t, T, H, D):
    """_rope_rows, with the contiguous case first."""
    if t.stride() == (H * D, D, 1) and t.shape == (T, H, D) and t.dtype is like.dtype and \
            t.get_device() == like.get_device():
        return H * D
    return _rope_rows(where, like, t, T, H, D)


def _same_strides(a, b):
    """Whether two arrays of one shape lie alike; a dimension of size 1 may
    carry any stride."""
    return a.stride() == b.stride() or all(n == 1 or x == y for n, x, y in zip(a.shape, a.stride(), b.stride()))


def _slot_array(where, t, other, dtype, shape, dev):
    """Strides of a number for each slot and head; `other` (or None) lies alike."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _need(where, False)
    if other is not None and other is not t and (other.dtype is not dtype or other.shape != shape or
                                                 other.get_device() != dev or not _same_strides(t, other)):
        _need(where, False)
    return t.stride()


_NO_STRIDES = (0, 0, 0)


def _cache(where, k_cache, v_cache, block_table, kv_len, k_exp, v_exp, weight, weight_out, pos, pos_out):
    """The cache of a call as thd_kv_cache's bytes, its B, Hkv, D and slots of
    a table's row, and the device."""
    import torch
    dev = _current(where, k_cache)
    shape, dtype, i32 = k_cache.shape, k_cache.dtype, torch.int32
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype is not dtype or v_cache.get_device() != dev or \
            not _same_strides(k_cache, v_cache):
        _need(where, False)
    e4m3 = dtype is torch.float8_e4m3fn
    if not e4m3 and dtype is not torch.bfloat16:
        raise ThdError(where, THD_ERR_UNSUPPORTED)
    pages, slots, heads, D = shape
    s0, s1, s2, s3 = k_cache.stride()
    if s3 != 1 or block_table.dim() != 2 or block_table.dtype is not i32 or block_table.get_device() != dev:
        _need(where, False)
    if pages == 1:
        s0 = 0
    if slots == 1:
        s1 = 0
    if heads == 1:
        s2 = 0
    B, max_pages = block_table.shape
    ts0, ts1 = block_table.stride()
    if not (ts1 == 1 or max_pages <= 1) or not (B <= 1 or ts0 == 0 or ts0 >= max_pages) or kv_len.dtype is not i32 or \
            kv_len.shape != (B,) or not kv_len.is_contiguous() or kv_len.get_device() != dev:
        _need(where, False)
    numbers = (pages, slots, heads)
    es = ws = ps = _NO_STRIDES
    ke = ve = 0
    if e4m3:
        if k_exp is None or v_exp is None:
            _need(where, False)
        es = _slot_array(where, k_exp, v_exp, torch.uint8, numbers, dev)
        ke, ve = k_exp.data_ptr(), v_exp.data_ptr()
    elif k_exp is not None or v_exp is not None:
        _need(where, False)
    if weight is not None:
        ws = _slot_array(where, weight, weight_out, torch.float32, numbers, dev)
    if pos is not None:
        ps = _slot_array(where, pos, pos_out, i32, numbers, dev)
    try:
        c = _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), ke, ve, block_table.data_ptr(), kv_len.data_ptr(), pages,
                        ts0, s0, s1, s2, *es, *ws, *ps, slots, max_pages, B, heads, D,
                        THD_DTYPE_E4M3 if e4m3 else THD_DTYPE_BF16)
    except struct.error:  # a size past the struct's
        _need(where, False)
    return c, B, heads, D, max_pages * slots, dev


def _numbers(where, t, n, dtype, dev):
    """A contiguous array of a call."""
    if t.dtype is not dtype or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        _need(where, False)


@functools.lru_cache(maxsize=1024)
def _sizes(library, name, *sizes):
    """A workspace's size, which goes by the sizes alone."""
    return getattr(library, name)(*sizes)


def _given_workspace(where, t, dev):
    if t.get_device() != dev or not t.is_contiguous():
        _need(where, False)
    return t.numel() * t.element_size()


def cache_append(k, v, k_cache, v_cache, block_table, kv_len, *, cu_seqlens=None, k_exp=None, v_exp=None, weight=None,
                 pos=None, tokens_seen=None, dev_status=None, stream=None):
    """New rows k, v [T, Hkv, D] bf16 (slices of a fused projection may be
    given) into the caches [num_pages, page_size, Hkv, D] (bf16 or
    float8_e4m3fn with uint8 exponents k_exp, v_exp [num_pages, page_size,
    Hkv]; any order of the first three dimensions in memory) at the pages of
    block_table int32 [B, max_pages]: sequence b's rows cu_seqlens[b] ..
    cu_seqlens[b + 1] (None: one row each) become its slots up to kv_len[b],
    which counts them.  weight fp32 and pos int32 (arrays like the exponents)
    are set for the new slots: 0, and the tokens' numbers up to tokens_seen[b]
    (None: kv_len).  Returns dev_status, which is only ever raised: pass one
    word to many calls, zeroed once."""
    import torch
    w = "thd_cache_append"
    c, B, Hkv, D, _, dev = _cache(w, k_cache, v_cache, block_table, kv_len, k_exp, v_exp, weight, None, pos, None)
    if k.dim() != 3 or k.dtype is not torch.bfloat16 or k.get_device() != dev:
        _need(w, False)
    T = k.shape[0]
    s_k, s_v = _row_stride(w, k, k, T, Hkv, D), _row_stride(w, k, v, T, Hkv, D)
    i32 = torch.int32
    if cu_seqlens is not None:
        _numbers(w, cu_seqlens, B + 1, i32, dev)
    if tokens_seen is not None:
        _numbers(w, tokens_seen, B, i32, dev)
    if dev_status is not None:
        _numbers(w, dev_status, 1, i32, dev)
    side = _aside(stream)
    st = dev_status
    if st is None:
        with _alloc_on(side):
            st = torch.zeros(1, dtype=i32, device=k.device)
    _check(w, thd_cache_append(c, k, v, s_k, s_v, T, cu_seqlens, weight, pos, tokens_seen, st, stream))
    if side is not None:
        _keep(side, stream, (k, v, k_cache, v_cache, block_table, kv_len, cu_seqlens, k_exp, v_exp, weight, pos, tokens_seen,
                             dev_status), (st,))
    return st


def attn_decode(q, k_cache, v_cache, block_table, kv_len, *, k_exp=None, v_exp=None, softmax_scale=None, softcap=0.0,
                dist_slopes=None, kv_start=None, pos=None, tokens_seen=None, weight=None, weight_out=None, out=None,
                lse=None, dev_status=None, workspace=None, stream=None):
    """Attention of one new token a sequence, q [B, Hq, D] bf16 (rows may be
    slices of a fused projection), over a cache as cache_append's; softcap and
    dist_slopes as attn_score_fwd's (distances by pos and tokens_seen, or by
    slots and kv_len), kv_start int32 [B] the first visible slot (a document's
    start while slots lie in order: not after cache_evict).  weight: the
    tokens' attention weights are added to it (into weight_out, if given).
    Returns (o [B, Hq, D], lse [Hq, B], dev_status)."""
    import torch
    w = "thd_attn_decode"
    if weight_out is None:
        weight_out = weight
    c, B, Hkv, D, capacity, dev = _cache(w, k_cache, v_cache, block_table, kv_len, k_exp, v_exp, weight, weight_out, pos,
                                         None)
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if (weight is None) != (weight_out is None) or q.dim() != 3 or q.dtype is not bf16 or q.get_device() != dev:
        _need(w, False)
    Hq = q.shape[1]
    s_q = _row_stride(w, q, q, B, Hq, D)
    if dev_status is not None:
        _numbers(w, dev_status, 1, i32, dev)
    if dist_slopes is not None:
        _numbers(w, dist_slopes, Hq, f32, dev)
    if kv_start is not None:
        _numbers(w, kv_start, B, i32, dev)
    if tokens_seen is not None:
        _numbers(w, tokens_seen, B, i32, dev)
    for t, n, dtype in ((out, (B, Hq, D), bf16), (lse, (Hq, B), f32)) if out is not None or lse is not None else ():
        if t is not None and (t.dtype is not dtype or t.shape != n or t.get_device() != dev or not t.is_contiguous()):
            _need(w, False)
    size = None if workspace is None else _given_workspace(w, workspace, dev)
    scale = 1.0 / math.sqrt(D) if softmax_scale is None else float(softmax_scale)
    side = _aside(stream)
    given = None if side is None else (q, k_cache, v_cache, block_table, kv_len, k_exp, v_exp, dist_slopes, kv_start, pos,
                                       tokens_seen, weight, weight_out, out, lse, dev_status, workspace)
    at = q.device
    with _alloc_on(side):
        o = torch.empty((B, Hq, D), dtype=bf16, device=at) if out is None else out
        l = torch.empty((Hq, B), dtype=f32, device=at) if lse is None else lse
        st = torch.zeros(1, dtype=i32, device=at) if dev_status is None else dev_status
        if size is None:
            size = _sizes(lib(), "thd_decode_workspace_size", B, Hq, Hkv, D, capacity, weight is not None)
            workspace = torch.empty(size, dtype=torch.uint8, device=at)
    _check(w, thd_attn_decode(c, q, s_q, o, l, Hq, scale, softcap, dist_slopes, kv_start, pos, tokens_seen, weight,
                              weight_out, workspace, size, st, stream))
    if side is not None:
        _keep(side, stream, given, (o, l, st))
    return o, l, st


def cache_evict(k_cache, v_cache, block_table, kv_len, weight, pos, tokens_seen, *, budget, sinks=0, recent=0,
                k_exp=None, v_exp=None, weight_out=None, pos_out=None, new_len=None, dev_status=None, workspace=None,
                stream=None):
    """Shrinks caches as cache_append's to `budget` slots a sequence and kv
    head: the first `sinks` and the last `recent` tokens stay (by pos and
    tokens_seen; the newest of them, where the budget holds fewer), then the
    largest weights.  Slots move in place; weight and
    pos too, unless weight_out, pos_out take them.  No kv_start of attn_decode
    means a document after that: give slots that no later token may see a weight
    of NaN and sinks 0, then they leave first, and all of them where a sequence
    has `budget` others.  Returns (new_len int32 [B], dev_status)."""
    import torch
    w = "thd_cache_evict"
    weight_out = weight if weight_out is None else weight_out
    pos_out = pos if pos_out is None else pos_out
    _need(w, weight is not None and pos is not None)
    c, B, Hkv, _, capacity, dev = _cache(w, k_cache, v_cache, block_table, kv_len, k_exp, v_exp, weight, weight_out, pos,
                                         pos_out)
    i32 = torch.int32
    _need(w, tokens_seen is not None)
    _numbers(w, tokens_seen, B, i32, dev)
    if new_len is not None:
        _numbers(w, new_len, B, i32, dev)
    if dev_status is not None:
        _numbers(w, dev_status, 1, i32, dev)
    size = None if workspace is None else _given_workspace(w, workspace, dev)
    side = _aside(stream)
    given = None if side is None else (k_cache, v_cache, block_table, kv_len, weight, pos, tokens_seen, k_exp, v_exp,
                                       weight_out, pos_out, new_len, dev_status, workspace)
    at = k_cache.device
    with _alloc_on(side):
        n = torch.empty(B, dtype=i32, device=at) if new_len is None else new_len
        st = torch.zeros(1, dtype=i32, device=at) if dev_status is None else dev_status
        if size is None:
            size = _sizes(lib(), "thd_evict_workspace_size", B, Hkv, capacity, budget)
            workspace = torch.empty(size, dtype=torch.uint8, device=at)
    _check(w, thd_cache_evict(c, weight, weight_out, pos, pos_out, tokens_seen, budget, sinks, recent, n, workspace,
                              size, st, stream))
    if side is not None:
        _keep(side, stream, given, (n, st))
    return n, st
