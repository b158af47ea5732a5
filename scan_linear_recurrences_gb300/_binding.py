"""ctypes binding of libmgscan (include/mgscan.h).

Argument marshalling only: every function here converts tensors/ints to raw
pointers and sizes and calls the C entry point of the same name.  All
arithmetic runs in the CUDA library; if the library is missing the call raises
instead of computing anything another way.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmgscan.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "mgscan.h")

MGS_OK = 0
MGS_ERR_INVALID_ARG = 1
MGS_ERR_UNSUPPORTED = 2
MGS_ERR_WORKSPACE = 3
MGS_ERR_CUDA = 4
MGS_ERR_TIMEOUT = 5
STATUS_NAMES = {0: "MGS_OK", 1: "MGS_ERR_INVALID_ARG", 2: "MGS_ERR_UNSUPPORTED",
                3: "MGS_ERR_WORKSPACE", 4: "MGS_ERR_CUDA", 5: "MGS_ERR_TIMEOUT"}

MGS_OP_MATRIX_AFFINE_SCAN_FWD = 1
MGS_OP_MATRIX_AFFINE_SCAN_BWD = 2
MGS_OP_MATRIX_SCAN_FWD = 3
MGS_OP_MATRIX_SCAN_BWD = 4
MGS_OP_PARALLEL_SCAN_LOG_FWD = 5
MGS_OP_PARALLEL_SCAN_LOG_BWD = 6
MGS_OP_LINEAR_SCAN_FWD = 7
MGS_OP_LINEAR_SCAN_BWD = 8
MGS_OP_GIVENS_AFFINE_SCAN_FWD = 9
MGS_OP_GIVENS_AFFINE_SCAN_BWD = 10
MGS_OP_GIVENS_MATRIX_SCAN_FWD = 11
MGS_OP_GIVENS_MATRIX_SCAN_BWD = 12
MGS_OP_DELTA_SCAN_FWD = 13
MGS_OP_MATRIX_AFFINE_SCAN_BWD_RECOMPUTE = 14

MGS_F32 = 0
MGS_BF16 = 1
MGS_I32 = 2
MGS_I64 = 3
GATED_SPAN = 64  # MGS_GATED_SPAN in include/mgscan.h
EXCHANGE_BLOCKS, EXCHANGE_ROUNDS = 8, 6  # MGS_EXCHANGE_BLOCKS, MGS_EXCHANGE_ROUNDS


class MGSError(RuntimeError):
    """A libmgscan entry point returned a status other than MGS_OK."""

    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")
        self.status = status


_lock = threading.Lock()
_lib = None
_torch_c = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_sz = ctypes.c_size_t
_flt = ctypes.c_float
_SIGNATURES = {
    "mgs_workspace_size": (_sz, [_int, _i64, _i64, _i64, _int]),
    "mgs_matrix_affine_scan_fwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_matrix_affine_scan_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_matrix_affine_scan_bwd_recompute": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp,
                                                    _sz, _vp]),
    "mgs_matrix_scan_fwd": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_matrix_scan_fwd_noalloc": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp]),
    "mgs_matrix_scan_bwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_parallel_scan_log_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "mgs_parallel_scan_log_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "mgs_linear_scan_fwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "mgs_linear_scan_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]),
    "mgs_givens_affine_scan_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_givens_affine_scan_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int,
                                          _vp, _sz, _vp]),
    "mgs_givens_matrix_scan_fwd": (_int, [_vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_givens_matrix_scan_bwd": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_delta_scan_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_linear_attention_workspace_size": (_sz, [_vp, _int]),
    "mgs_linear_attention_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mgs_linear_attention_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                        _vp]),
    "mgs_linear_attention_step": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "mgs_rms_norm_fwd": (_int, [_vp, _vp, _vp, _flt, _vp, _vp, _vp, _i64, _i64, _int, _vp]),
    "mgs_rms_norm_fp8_fwd": (_int, [_vp, _vp, _vp, _flt, _vp, _vp, _vp, _i64, _i64, _int, _int, _vp]),
    "mgs_rms_norm_bwd_workspace_size": (_sz, [_i64, _i64]),
    "mgs_rms_norm_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_clip_grad_norm_workspace_size": (_sz, [_i64]),
    "mgs_clip_grad_norm": (_int, [_vp, _vp, _vp, _vp, _i64, _flt, _vp, _vp, _sz, _vp]),
    "mgs_gated_scan_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mgs_gated_scan_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mgs_gated_scan_step": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "mgs_qk_norm_fwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mgs_qk_norm_bwd_workspace_size": (_sz, [_vp]),
    "mgs_qk_norm_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "mgs_embedding_fwd": (_int, [_vp, _int, _vp, _flt, _vp, _i64, _i64, _i64, _int, _vp]),
    "mgs_embedding_bwd_workspace_size": (_sz, [_i64, _i64, _i64]),
    "mgs_embedding_bwd": (_int, [_vp, _int, _vp, _i64, _flt, _vp, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "mgs_check": (_int, [_vp]),
    "mgs_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
    "mgs_debug_wait_flag": (_int, [_vp, _vp]),
    "mgs_debug_exchange": (_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64, _vp, _vp, _vp]),
    "mgs_status_string": (ctypes.c_char_p, [_int]),
    "mgs_version": (_int, []),
}


def lib():
    """The loaded CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with scan_linear_recurrences_gb300.build.build() "
                    "(nvcc, sm_103a); there is no other implementation to fall back to")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def exported_symbols():
    """Names declared in the C header (used to check the library's exports)."""
    return list(_SIGNATURES)


def _ptr(x):
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:  # an address
        return x


def _stream(s):
    global _torch_c
    if s is None:
        if _torch_c is None:
            import torch
            _torch_c = torch._C
        return _torch_c._cuda_getCurrentRawStream(_torch_c._cuda_getDevice())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _call(name, *args):
    st = getattr(_lib or lib(), name)(*args)
    if st != MGS_OK:
        raise MGSError(name, st)
    return st


# ---------------------------------------------------------------- raw entry points
def mgs_workspace_size(op, B, T, H_or_D, k):
    return int(lib().mgs_workspace_size(op, B, T, H_or_D, k))


def mgs_matrix_affine_scan_fwd(A, b, h0, h, B, T, H, k, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_matrix_affine_scan_fwd", _ptr(A), _ptr(b), _ptr(h0), _ptr(h), B, T, H, k,
                 _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_matrix_affine_scan_bwd(A, h0, h, grad_h, dA, db, dh0, B, T, H, k, workspace=None,
                               workspace_bytes=0, stream=None):
    return _call("mgs_matrix_affine_scan_bwd", _ptr(A), _ptr(h0), _ptr(h), _ptr(grad_h), _ptr(dA),
                 _ptr(db), _ptr(dh0), B, T, H, k, _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_matrix_affine_scan_bwd_recompute(A, b, h0, grad_h, dA, db, dh0, B, T, H, k, workspace=None,
                                         workspace_bytes=0, stream=None):
    return _call("mgs_matrix_affine_scan_bwd_recompute", _ptr(A), _ptr(b), _ptr(h0), _ptr(grad_h), _ptr(dA),
                 _ptr(db), _ptr(dh0), B, T, H, k, _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_matrix_scan_fwd(A, P, B, T, H, k, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_matrix_scan_fwd", _ptr(A), _ptr(P), B, T, H, k, _ptr(workspace), workspace_bytes,
                 _stream(stream))


def mgs_matrix_scan_fwd_noalloc(A, P, B, T, H, k, stream=None):
    """matrix_scan forward using the library's built-in device scratch; for
    callers that cannot allocate device memory (see include/mgscan.h)."""
    return _call("mgs_matrix_scan_fwd_noalloc", _ptr(A), _ptr(P), B, T, H, k, _stream(stream))


NOALLOC_SCRATCH_BYTES = 4 << 20  # MGS_NOALLOC_SCRATCH_BYTES in include/mgscan.h


def mgs_matrix_scan_bwd(A, P, grad_P, dA, B, T, H, k, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_matrix_scan_bwd", _ptr(A), _ptr(P), _ptr(grad_P), _ptr(dA), B, T, H, k,
                 _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_parallel_scan_log_fwd(log_coeffs, log_values, log_h0, h, log_h, B, T, D, workspace=None,
                              workspace_bytes=0, stream=None):
    return _call("mgs_parallel_scan_log_fwd", _ptr(log_coeffs), _ptr(log_values), _ptr(log_h0), _ptr(h),
                 _ptr(log_h), B, T, D, _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_parallel_scan_log_bwd(log_coeffs, log_values, log_h0, h, grad_h, d_log_coeffs, d_log_values,
                              d_log_h0, B, T, D, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_parallel_scan_log_bwd", _ptr(log_coeffs), _ptr(log_values), _ptr(log_h0), _ptr(h),
                 _ptr(grad_h), _ptr(d_log_coeffs), _ptr(d_log_values), _ptr(d_log_h0), B, T, D,
                 _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_linear_scan_fwd(a, b, h0, h, B, T, D, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_linear_scan_fwd", _ptr(a), _ptr(b), _ptr(h0), _ptr(h), B, T, D, _ptr(workspace),
                 workspace_bytes, _stream(stream))


def mgs_linear_scan_bwd(a, h0, h, grad_h, da, db, dh0, B, T, D, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_linear_scan_bwd", _ptr(a), _ptr(h0), _ptr(h), _ptr(grad_h), _ptr(da), _ptr(db), _ptr(dh0),
                 B, T, D, _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_givens_affine_scan_fwd(theta, a, b, h0, h, B, T, H, k, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_givens_affine_scan_fwd", _ptr(theta), _ptr(a), _ptr(b), _ptr(h0), _ptr(h), B, T, H, k,
                 _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_givens_affine_scan_bwd(theta, a, h0, h, grad_h, d_theta, da, db, dh0, B, T, H, k, workspace=None,
                               workspace_bytes=0, stream=None):
    return _call("mgs_givens_affine_scan_bwd", _ptr(theta), _ptr(a), _ptr(h0), _ptr(h), _ptr(grad_h),
                 _ptr(d_theta), _ptr(da), _ptr(db), _ptr(dh0), B, T, H, k, _ptr(workspace), workspace_bytes,
                 _stream(stream))


def mgs_givens_matrix_scan_fwd(theta, P, B, T, H, k, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_givens_matrix_scan_fwd", _ptr(theta), _ptr(P), B, T, H, k, _ptr(workspace),
                 workspace_bytes, _stream(stream))


def mgs_givens_matrix_scan_bwd(theta, P, grad_P, d_theta, B, T, H, k, workspace=None, workspace_bytes=0,
                               stream=None):
    return _call("mgs_givens_matrix_scan_bwd", _ptr(theta), _ptr(P), _ptr(grad_P), _ptr(d_theta), B, T, H, k,
                 _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_delta_scan_fwd(q, k, v, beta, S0, o, S_T, B, T, H, D, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_delta_scan_fwd", _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T),
                 B, T, H, D, _ptr(workspace), workspace_bytes, _stream(stream))


_ATTENTION_SHAPE = struct.Struct("<4q3if15q")
_NO_STRIDES = (0, 0, 0)


def mgs_attention_shape(B, T, H, Hk, D, dtype, fixed_decay, scale, q_stride, k_stride, v_stride,
                        g_stride=_NO_STRIDES, do_stride=_NO_STRIDES):
    """The C struct of that name, as bytes.  Strides: (batch, step, head) in elements."""
    return _ATTENTION_SHAPE.pack(B, T, H, Hk, D, dtype, fixed_decay, scale, *q_stride, *k_stride, *v_stride,
                                 *g_stride, *do_stride)


def mgs_linear_attention_workspace_size(shape, backward):
    return int(lib().mgs_linear_attention_workspace_size(shape, int(backward)))


def mgs_linear_attention_fwd(shape, q, k, v, g, S0, o, S_T, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_linear_attention_fwd", shape, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(o), _ptr(S_T),
                 _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_linear_attention_bwd(shape, q, k, v, g, S0, grad_o, grad_S_T, dq, dk, dv, dg, dS0, workspace=None,
                             workspace_bytes=0, stream=None):
    return _call("mgs_linear_attention_bwd", shape, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S0), _ptr(grad_o),
                 _ptr(grad_S_T), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dS0), _ptr(workspace), workspace_bytes,
                 _stream(stream))


def mgs_linear_attention_step(shape, q, k, v, g, S, slots, n_slots, o, stream=None):
    return _call("mgs_linear_attention_step", shape, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(S), _ptr(slots),
                 n_slots, _ptr(o), _stream(stream))


def mgs_rms_norm_fwd(x, residual, weight, eps, r, y, rstd, rows, N, dtype, stream=None):
    return _call("mgs_rms_norm_fwd", _ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(r), _ptr(y), _ptr(rstd), rows,
                 N, dtype, _stream(stream))


def mgs_rms_norm_fp8_fwd(x, residual, weight, eps, r, q, scales, rows, N, group, dtype, stream=None):
    return _call("mgs_rms_norm_fp8_fwd", _ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(r), _ptr(q), _ptr(scales),
                 rows, N, group, dtype, _stream(stream))


def mgs_rms_norm_bwd_workspace_size(rows, N):
    return int(lib().mgs_rms_norm_bwd_workspace_size(rows, N))


def mgs_rms_norm_bwd(r, weight, rstd, grad_y, grad_r, dx, dweight, rows, N, dtype, workspace=None, workspace_bytes=0,
                     stream=None):
    return _call("mgs_rms_norm_bwd", _ptr(r), _ptr(weight), _ptr(rstd), _ptr(grad_y), _ptr(grad_r), _ptr(dx),
                 _ptr(dweight), rows, N, dtype, _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_clip_grad_norm_workspace_size(count):
    return int(lib().mgs_clip_grad_norm_workspace_size(count))


def mgs_clip_grad_norm(grads, outs, numels, dtypes, max_norm, norm, workspace=None, workspace_bytes=0, stream=None):
    """grads, outs: lists of device addresses; numels, dtypes: lists of ints."""
    n = len(grads)
    return _call("mgs_clip_grad_norm", struct.pack(f"{n}Q", *grads), struct.pack(f"{n}Q", *outs),
                 struct.pack(f"{n}q", *numels), struct.pack(f"{n}i", *dtypes), n, max_norm, _ptr(norm),
                 _ptr(workspace), workspace_bytes, _stream(stream))


_GATED_SHAPE = struct.Struct("<3q2i6q")


def mgs_gated_shape(B, T, D, dtype, positive, gate_stride, value_stride, gh_stride=(0, 0)):
    """The C struct of that name, as bytes.  Strides: (batch, step) in elements."""
    return _GATED_SHAPE.pack(B, T, D, dtype, positive, *gate_stride, *value_stride, *gh_stride)


def mgs_gated_scan_fwd(shape, gate, value, h0, h, h_T, carries, stream=None):
    return _call("mgs_gated_scan_fwd", shape, _ptr(gate), _ptr(value), _ptr(h0), _ptr(h), _ptr(h_T), _ptr(carries),
                 _stream(stream))


def mgs_gated_scan_bwd(shape, gate, value, carries, grad_h, grad_h_T, d_gate, d_value, d_h0, stream=None):
    return _call("mgs_gated_scan_bwd", shape, _ptr(gate), _ptr(value), _ptr(carries), _ptr(grad_h), _ptr(grad_h_T),
                 _ptr(d_gate), _ptr(d_value), _ptr(d_h0), _stream(stream))


def mgs_gated_scan_step(shape, gate, value, state, slots, n_slots, h, stream=None):
    return _call("mgs_gated_scan_step", shape, _ptr(gate), _ptr(value), _ptr(state), _ptr(slots), n_slots, _ptr(h),
                 _stream(stream))


_QK_NORM_SHAPE = struct.Struct("<5q4if4x14q")


def mgs_qk_norm_shape(B, T, Hq, Hk, positions, D, dtype, rotary, interleaved, eps, q_stride, k_stride,
                      gq_stride=_NO_STRIDES, gk_stride=_NO_STRIDES, pos_stride=(0, 0)):
    """The C struct of that name, as bytes.  Strides: (batch, step, head), positions (batch, step), in elements."""
    return _QK_NORM_SHAPE.pack(B, T, Hq, Hk, positions, D, dtype, rotary, interleaved, eps, *q_stride, *k_stride,
                               *gq_stride, *gk_stride, *pos_stride)


def mgs_qk_norm_fwd(shape, q, k, q_weight, k_weight, table, token_positions, yq, yk, stream=None):
    return _call("mgs_qk_norm_fwd", shape, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(table),
                 _ptr(token_positions), _ptr(yq), _ptr(yk), _stream(stream))


def mgs_qk_norm_bwd_workspace_size(shape):
    return int(lib().mgs_qk_norm_bwd_workspace_size(shape))


def mgs_qk_norm_bwd(shape, q, k, q_weight, k_weight, grad_yq, grad_yk, table, token_positions, dq, dk, dq_weight,
                    dk_weight, workspace=None, workspace_bytes=0, stream=None):
    return _call("mgs_qk_norm_bwd", shape, _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(grad_yq),
                 _ptr(grad_yk), _ptr(table), _ptr(token_positions), _ptr(dq), _ptr(dk), _ptr(dq_weight),
                 _ptr(dk_weight), _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_embedding_fwd(tokens, token_type, weight, scale, out, N, V, D, dtype, stream=None):
    return _call("mgs_embedding_fwd", _ptr(tokens), token_type, _ptr(weight), scale, _ptr(out), N, V, D, dtype,
                 _stream(stream))


def mgs_embedding_bwd_workspace_size(N, V, D):
    return int(lib().mgs_embedding_bwd_workspace_size(N, V, D))


def mgs_embedding_bwd(tokens, token_type, grad, grad_stride, scale, dweight, N, V, D, dtype, workspace=None,
                      workspace_bytes=0, stream=None):
    return _call("mgs_embedding_bwd", _ptr(tokens), token_type, _ptr(grad), grad_stride, scale, _ptr(dweight), N, V, D,
                 dtype, _ptr(workspace), workspace_bytes, _stream(stream))


def mgs_check(stream=None):
    return _call("mgs_check", _stream(stream))


def mgs_set_wait_timeout_ns(ns: int):
    lib().mgs_set_wait_timeout_ns(int(ns))


def mgs_debug_wait_flag(flag, stream=None):
    return _call("mgs_debug_wait_flag", _ptr(flag), _stream(stream))


def mgs_debug_exchange(late_block, late_round, late_ns, rounds, wrong, stream=None):
    return _call("mgs_debug_exchange", late_block, late_round, late_ns, _ptr(rounds), _ptr(wrong), _stream(stream))


def mgs_status_string(status: int) -> str:
    return lib().mgs_status_string(status).decode()


def mgs_version() -> int:
    return int(lib().mgs_version())
