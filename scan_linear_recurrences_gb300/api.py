"""Tensor-level API over the C ABI: shape checks, output/workspace allocation
with torch (device memory is torch's job here), then one libmgscan call.

Also provides ``torch.autograd.Function`` wrappers whose forward and backward
are the library's fwd/bwd entry points, for use inside models.

``stream``: the kernels' stream (a torch stream or its address; None: the current
one).  The caller orders it after the work that makes the inputs, and after what
torch's current stream has been given: outputs are allocated there.
"""
from __future__ import annotations

import contextlib
import operator

import torch
from torch.autograd.function import once_differentiable

from . import _binding as _b


def _check(t, name, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (the library runs only on the GPU)")
    if t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _on(stream, device):
    """The context in which memory and copies belong to the call's stream (an address, a torch stream, or None: the
    current one).  What is allocated in it may be dropped when the call returns: it goes back to that stream."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):  # address 0: the default stream, for which torch has no external one
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _scratch(n, device, stream):
    """n bytes of workspace that stay reserved until `stream` is done with them."""
    if not n:
        return None
    with _on(stream, device):
        return torch.empty(n, dtype=torch.uint8, device=device)


def workspace(op, B, T, H_or_D, k, device, stream=None):
    """A workspace tensor of the size the op needs (None when it needs none), of the stream that it is for."""
    n = _b.mgs_workspace_size(op, B, T, H_or_D, k)
    return _scratch(n, device, stream), n


# ---------------------------------------------------------------- matrix_affine_scan
def matrix_affine_scan_fwd(A, b, h0=None, out=None, stream=None):
    """h_t = A_t h_{t-1} + b_t.  A [B,T,H,k,k], b [B,T,H,k], h0 [B,H,k] or None."""
    B, T, H, k = b.shape
    _check(A, "A", (B, T, H, k, k)); _check(b, "b")
    if h0 is not None:
        _check(h0, "h0", (B, H, k))
    h = out if out is not None else torch.empty_like(b)
    ws, nws = workspace(_b.MGS_OP_MATRIX_AFFINE_SCAN_FWD, B, T, H, k, b.device, stream)
    _b.mgs_matrix_affine_scan_fwd(A, b, h0, h, B, T, H, k, ws, nws, stream)
    return h


def matrix_affine_scan_bwd(A, h0, h, grad_h, need_dh0=True, stream=None):
    """Returns (dA, db, dh0) for L = sum <grad_h, h>; dh0 is None unless requested."""
    B, T, H, k = h.shape
    _check(A, "A", (B, T, H, k, k)); _check(h, "h"); _check(grad_h, "grad_h", (B, T, H, k))
    if h0 is not None:
        _check(h0, "h0", (B, H, k))
    dA = torch.empty_like(A)
    db = torch.empty_like(h)
    dh0 = torch.empty((B, H, k), dtype=torch.float32, device=h.device) if need_dh0 else None
    ws, nws = workspace(_b.MGS_OP_MATRIX_AFFINE_SCAN_BWD, B, T, H, k, h.device, stream)
    _b.mgs_matrix_affine_scan_bwd(A, h0, h, grad_h, dA, db, dh0, B, T, H, k, ws, nws, stream)
    return dA, db, dh0


def matrix_affine_scan_bwd_recompute(A, b, h0, grad_h, need_dh0=True, stream=None):
    """The same gradients as matrix_affine_scan_bwd without the saved h: the
    call recomputes the forward from A, b and h0 (checkpoints in a workspace)."""
    B, T, H, k = b.shape
    _check(A, "A", (B, T, H, k, k)); _check(b, "b"); _check(grad_h, "grad_h", (B, T, H, k))
    if h0 is not None:
        _check(h0, "h0", (B, H, k))
    dA = torch.empty_like(A)
    db = torch.empty_like(b)
    dh0 = torch.empty((B, H, k), dtype=torch.float32, device=b.device) if need_dh0 else None
    ws, nws = workspace(_b.MGS_OP_MATRIX_AFFINE_SCAN_BWD_RECOMPUTE, B, T, H, k, b.device, stream)
    _b.mgs_matrix_affine_scan_bwd_recompute(A, b, h0, grad_h, dA, db, dh0, B, T, H, k, ws, nws, stream)
    return dA, db, dh0


# ---------------------------------------------------------------- matrix_scan
def matrix_scan_fwd(A, out=None, stream=None):
    """P_t = A_t P_{t-1}, P_0 = I.  A [B,T,H,k,k]."""
    B, T, H, k, _ = A.shape
    _check(A, "A", (B, T, H, k, k))
    P = out if out is not None else torch.empty_like(A)
    ws, nws = workspace(_b.MGS_OP_MATRIX_SCAN_FWD, B, T, H, k, A.device, stream)
    _b.mgs_matrix_scan_fwd(A, P, B, T, H, k, ws, nws, stream)
    return P


def matrix_scan_bwd(A, P, grad_P, stream=None):
    B, T, H, k, _ = A.shape
    _check(A, "A", (B, T, H, k, k)); _check(P, "P", A.shape); _check(grad_P, "grad_P", A.shape)
    dA = torch.empty_like(A)
    ws, nws = workspace(_b.MGS_OP_MATRIX_SCAN_BWD, B, T, H, k, A.device, stream)
    _b.mgs_matrix_scan_bwd(A, P, grad_P, dA, B, T, H, k, ws, nws, stream)
    return dA


# ---------------------------------------------------------------- parallel_scan_log
def parallel_scan_log_fwd(log_coeffs, log_values, log_h0=None, want_log=False, stream=None):
    """Heinsen log-space scan; returns h (and log h when want_log)."""
    B, T, D = log_coeffs.shape
    _check(log_coeffs, "log_coeffs"); _check(log_values, "log_values", (B, T, D))
    if log_h0 is not None:
        _check(log_h0, "log_h0", (B, D))
    h = torch.empty_like(log_coeffs)
    lh = torch.empty_like(log_coeffs) if want_log else None
    _b.mgs_parallel_scan_log_fwd(log_coeffs, log_values, log_h0, h, lh, B, T, D, None, 0, stream)
    return (h, lh) if want_log else h


def parallel_scan_log_bwd(log_coeffs, log_values, log_h0, h, grad_h, stream=None):
    """Returns (d_log_coeffs, d_log_values, d_log_h0 or None).

    h is the saved forward output, or None to recompute it inside the call
    (checkpoints every 16 steps in a workspace of 4*B*ceil(T/16)*D bytes)."""
    B, T, D = log_coeffs.shape
    for t, n in ((log_coeffs, "log_coeffs"), (log_values, "log_values"), (grad_h, "grad_h")):
        _check(t, n, (B, T, D))
    if h is not None:
        _check(h, "h", (B, T, D))
    if log_h0 is not None:
        _check(log_h0, "log_h0", (B, D))
    dlc = torch.empty_like(log_coeffs)
    dlv = torch.empty_like(log_values)
    dl0 = torch.empty_like(log_h0) if log_h0 is not None else None
    ws, nws = (None, 0) if h is not None else \
        workspace(_b.MGS_OP_PARALLEL_SCAN_LOG_BWD, B, T, D, 0, log_coeffs.device, stream)
    _b.mgs_parallel_scan_log_bwd(log_coeffs, log_values, log_h0, h, grad_h, dlc, dlv, dl0, B, T, D,
                                 ws, nws, stream)
    return dlc, dlv, dl0


# ---------------------------------------------------------------- Givens-mesh scans
GIVENS_K = 8
GIVENS_N = GIVENS_K * (GIVENS_K - 1) // 2


def givens_affine_scan_fwd(theta, a, b, h0=None, stream=None):
    """h_t = G(theta_t) diag(a_t) h_{t-1} + b_t.  theta [B,T,H,28], a [B,T,H,8] or None,
    b [B,T,H,8], h0 [B,H,8] or None."""
    B, T, H, k = b.shape
    _check(theta, "theta", (B, T, H, k * (k - 1) // 2)); _check(b, "b")
    if a is not None:
        _check(a, "a", (B, T, H, k))
    if h0 is not None:
        _check(h0, "h0", (B, H, k))
    h = torch.empty_like(b)
    ws, nws = workspace(_b.MGS_OP_GIVENS_AFFINE_SCAN_FWD, B, T, H, k, b.device, stream)
    _b.mgs_givens_affine_scan_fwd(theta, a, b, h0, h, B, T, H, k, ws, nws, stream)
    return h


def givens_affine_scan_bwd(theta, a, h0, h, grad_h, need_dh0=True, stream=None):
    """Returns (d_theta, da or None, db, dh0 or None) for L = sum <grad_h, h>."""
    B, T, H, k = h.shape
    _check(theta, "theta", (B, T, H, k * (k - 1) // 2)); _check(h, "h"); _check(grad_h, "grad_h", (B, T, H, k))
    if a is not None:
        _check(a, "a", (B, T, H, k))
    if h0 is not None:
        _check(h0, "h0", (B, H, k))
    dth = torch.empty_like(theta)
    da = torch.empty_like(a) if a is not None else None
    db = torch.empty_like(h)
    dh0 = torch.empty((B, H, k), dtype=torch.float32, device=h.device) if need_dh0 else None
    ws, nws = workspace(_b.MGS_OP_GIVENS_AFFINE_SCAN_BWD, B, T, H, k, h.device, stream)
    _b.mgs_givens_affine_scan_bwd(theta, a, h0, h, grad_h, dth, da, db, dh0, B, T, H, k, ws, nws, stream)
    return dth, da, db, dh0


def givens_matrix_scan_fwd(theta, k=GIVENS_K, stream=None):
    """P_t = G(theta_t) P_{t-1}, P_0 = I.  theta [B,T,H,28] -> P [B,T,H,8,8]."""
    B, T, H, n = theta.shape
    _check(theta, "theta", (B, T, H, k * (k - 1) // 2))
    P = torch.empty((B, T, H, k, k), dtype=torch.float32, device=theta.device)
    ws, nws = workspace(_b.MGS_OP_GIVENS_MATRIX_SCAN_FWD, B, T, H, k, theta.device, stream)
    _b.mgs_givens_matrix_scan_fwd(theta, P, B, T, H, k, ws, nws, stream)
    return P


def givens_matrix_scan_bwd(theta, P, grad_P, stream=None):
    B, T, H, k, _ = P.shape
    _check(theta, "theta", (B, T, H, k * (k - 1) // 2)); _check(P, "P"); _check(grad_P, "grad_P", P.shape)
    dth = torch.empty_like(theta)
    ws, nws = workspace(_b.MGS_OP_GIVENS_MATRIX_SCAN_BWD, B, T, H, k, theta.device, stream)
    _b.mgs_givens_matrix_scan_bwd(theta, P, grad_P, dth, B, T, H, k, ws, nws, stream)
    return dth


# ---------------------------------------------------------------- delta rule
def delta_scan_fwd(q, k, v, beta, S0=None, want_state=False, stream=None):
    """DeltaNet's delta rule: S_t = S_{t-1} + beta_t (v_t - S_{t-1} k_t) k_t^T,
    o_t = S_t q_t.  q, k, v [B,T,H,64], beta [B,T,H], S0 [B,H,64,64] or None.
    Returns o (and the final state when want_state)."""
    B, T, H, D = q.shape
    _check(q, "q"); _check(k, "k", q.shape); _check(v, "v", q.shape); _check(beta, "beta", (B, T, H))
    if S0 is not None:
        _check(S0, "S0", (B, H, D, D))
    o = torch.empty_like(q)
    ST = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device) if want_state else None
    ws, nws = workspace(_b.MGS_OP_DELTA_SCAN_FWD, B, T, H, D, q.device, stream)
    _b.mgs_delta_scan_fwd(q, k, v, beta, S0, o, ST, B, T, H, D, ws, nws, stream)
    return (o, ST) if want_state else o


# ---------------------------------------------------------------- linear_scan
def linear_scan_fwd(a, b, h0=None, stream=None):
    """h_t = a_t * h_{t-1} + b_t elementwise.  a, b [B,T,D], h0 [B,D] or None."""
    B, T, D = a.shape
    _check(a, "a"); _check(b, "b", (B, T, D))
    if h0 is not None:
        _check(h0, "h0", (B, D))
    h = torch.empty_like(b)
    ws, nws = workspace(_b.MGS_OP_LINEAR_SCAN_FWD, B, T, D, 1, b.device, stream)
    _b.mgs_linear_scan_fwd(a, b, h0, h, B, T, D, ws, nws, stream)
    return h


def linear_scan_bwd(a, h0, h, grad_h, need_dh0=True, stream=None):
    """Returns (da, db, dh0 or None) for L = sum grad_h * h."""
    B, T, D = a.shape
    for t, n in ((a, "a"), (h, "h"), (grad_h, "grad_h")):
        _check(t, n, (B, T, D))
    if h0 is not None:
        _check(h0, "h0", (B, D))
    da, db = torch.empty_like(a), torch.empty_like(a)
    dh0 = torch.empty((B, D), dtype=torch.float32, device=a.device) if need_dh0 else None
    ws, nws = workspace(_b.MGS_OP_LINEAR_SCAN_BWD, B, T, D, 1, a.device, stream)
    _b.mgs_linear_scan_bwd(a, h0, h, grad_h, da, db, dh0, B, T, D, ws, nws, stream)
    return da, db, dh0


# ---------------------------------------------------------------- linear attention with a decay
_DTYPES = {torch.float32: _b.MGS_F32, torch.bfloat16: _b.MGS_BF16}


def _check_typed(t, name, shape, dtype, dense=True, device=None):
    """One CUDA tensor of this shape, type and device (None: any; a None dtype: fp32 or bf16)."""
    try:
        if (t.is_cuda and (dtype is t.dtype or dtype is None and t.dtype in _DTYPES)
                and (shape is None or t.shape == shape) and (not dense or t.is_contiguous())
                and (device is None or t.device == device)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (the library runs only on the GPU)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is None and t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}".replace("torch.", ""))
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _head_strides(t, name):
    """(batch, step, head) strides of [B,T,h,D] whose heads are contiguous."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return st[:-1]


def _apart(t, stream):
    """t, or a dense copy of a broadcast t: the tensor-core kernels load through tensor maps, which have no
    zero strides, and the copy costs less than the kernel without them."""
    st = t.stride()
    if 0 not in st or all(s or n <= 1 for s, n in zip(st, t.shape)):
        return t
    with _on(stream, t.device):
        return t.contiguous()


def _attention_shape(q, k, v, g, scale, stream, grad_o=None):
    """The checked arguments as the C struct, (B, T, H, Hk, D), and the tensors to pass."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B,T,Hk,D] tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("v must be a [B,T,H,D] tensor")
    (B, T, Hk, D), H, dev = q.shape, v.shape[2], q.device
    _check_typed(q, "q", None, None, dense=False)
    _check_typed(k, "k", q.shape, q.dtype, dense=False, device=dev)
    _check_typed(v, "v", (B, T, H, D), q.dtype, dense=False, device=dev)
    if Hk == 0 or H % Hk:
        raise ValueError(f"{Hk} query/key heads do not divide {H} value heads")
    if D not in (64, 128):
        raise ValueError(f"heads of {D}: 64 and 128 are supported")
    fixed = isinstance(g, torch.Tensor) and g.dim() == 1
    _check_typed(g, "g", (H,) if fixed else (B, T, H), torch.float32, dense=fixed, device=dev)
    if grad_o is not None:
        _check_typed(grad_o, "grad_o", v.shape, q.dtype, dense=False, device=dev)
    # (fp32 is read through dense tensors of its terms, but for the gradients' products of q with dq and k with dk)
    if q.dtype == torch.bfloat16 or grad_o is not None:
        q, k = _apart(q, stream), _apart(k, stream)
    if q.dtype == torch.bfloat16:
        v, grad_o = _apart(v, stream), _apart(grad_o, stream) if grad_o is not None else None
    shape = _b.mgs_attention_shape(
        B, T, H, Hk, D, _DTYPES[q.dtype], fixed, D ** -0.5 if scale is None else scale, _head_strides(q, "q"),
        _head_strides(k, "k"), _head_strides(v, "v"), (0, 0, 1) if fixed else g.stride(),
        _head_strides(grad_o, "grad_o") if grad_o is not None else (0, 0, 0))
    return shape, (B, T, H, Hk, D), (q, k, v, grad_o)


_increment_version = torch.autograd.graph.increment_version


def _written(tensors):
    """Marks tensors that a call has written in place, so that autograd notices where it had saved one of them."""
    try:
        _increment_version(tensors)
    except RuntimeError:  # inference tensors have no versions
        _increment_version([t for t in tensors if not t.is_inference()])


def linear_attention_fwd(q, k, v, g, S0=None, scale=None, want_state=False, stream=None):
    """Linear attention with a decay for each head:
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t (scale: D^-1/2 unless given).

    q, k [B,T,Hk,D], v [B,T,H,D] (fp32 or bf16, D 64 or 128, Hk dividing H: value head h reads query/key
    head h // (H // Hk); any strides of 16 bytes whose heads are contiguous), g [B,T,H] or [H] fp32 (the
    decay's logarithm; -inf starts the state anew), S0 [B,H,D,D] fp32 or None.  States and sums are fp32; bf16
    outputs are rounded once (relative error 1.7e-3), fp32 ones err by 2e-7 to 7e-7.
    Returns o [B,T,H,D] (and the final state when want_state)."""
    shape, (B, T, H, Hk, D), (q, k, v, _) = _attention_shape(q, k, v, g, scale, stream)
    if S0 is not None:
        _check_typed(S0, "S0", (B, H, D, D), torch.float32, device=q.device)
    o = torch.empty((B, T, H, D), dtype=q.dtype, device=q.device)
    ST = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device) if want_state else None
    n = _b.mgs_linear_attention_workspace_size(shape, 0)
    _b.mgs_linear_attention_fwd(shape, q, k, v, g, S0, o, ST, _scratch(n, q.device, stream), n, stream)
    return (o, ST) if want_state else o


def linear_attention_bwd(q, k, v, g, grad_o, S0=None, grad_ST=None, scale=None, stream=None):
    """Gradients of linear_attention_fwd for L = <grad_o, o> + <grad_ST, S_T>: returns (dq, dk, dv, dg, dS0),
    dS0 None without S0.  dg is [B,T,H], or [H] for a g of one decay a head."""
    shape, (B, T, H, Hk, D), (q, k, v, grad_o) = _attention_shape(q, k, v, g, scale, stream, grad_o)
    for t, name in ((S0, "S0"), (grad_ST, "grad_ST")):
        if t is not None:
            _check_typed(t, name, (B, H, D, D), torch.float32, device=q.device)
    dq = torch.empty((B, T, Hk, D), dtype=q.dtype, device=q.device)
    dk = torch.empty_like(dq)
    dv = torch.empty((B, T, H, D), dtype=q.dtype, device=q.device)
    dg = torch.empty(g.shape, dtype=torch.float32, device=q.device)
    dS0 = torch.empty_like(S0) if S0 is not None else None
    n = _b.mgs_linear_attention_workspace_size(shape, 1)
    _b.mgs_linear_attention_bwd(shape, q, k, v, g, S0, grad_o, grad_ST, dq, dk, dv, dg, dS0, _scratch(n, q.device, stream), n,
                                stream)
    return dq, dk, dv, dg, dS0


def linear_attention_step(q, k, v, g, S, slots=None, scale=None, out=None, stream=None):
    """One token of each of B sequences: q, k [B,Hk,D], v [B,H,D], g [B,H] or [H] fp32, the cache of states
    S [N,H,D,D] fp32, updated in place.  slots [B] int32: each sequence's place in the cache (None: b itself);
    a place outside 0..N-1 marks an empty row, whose output is 0.  Returns o [B,H,D]."""
    (B, Hk, D), H, dev = q.shape, v.shape[1], q.device
    dt = q.dtype
    _check_typed(q, "q", None, None, dense=False)
    _check_typed(k, "k", q.shape, dt, dense=False, device=dev)
    _check_typed(v, "v", (B, H, D), dt, dense=False, device=dev)
    if Hk == 0 or H % Hk:
        raise ValueError(f"{Hk} query/key heads do not divide {H} value heads")
    if D not in (64, 128):
        raise ValueError(f"heads of {D}: 64 and 128 are supported")
    fixed = g.dim() == 1
    _check_typed(g, "g", (H,) if fixed else (B, H), torch.float32, dense=fixed, device=dev)
    _check_typed(S, "S", (S.shape[0], H, D, D), torch.float32, device=dev)
    if slots is not None:
        _check_typed(slots, "slots", (B,), torch.int32, device=dev)
    elif S.shape[0] < B:
        raise ValueError(f"{B} sequences without slots need a cache of as many states, not {S.shape[0]}")
    written = (S,) if out is None else (S, out)
    if out is None:
        out = torch.empty((B, H, D), dtype=dt, device=dev)
    else:
        _check_typed(out, "out", (B, H, D), dt, device=dev)
    (qb, qh), (kb, kh), (vb, vh) = _head_strides(q, "q"), _head_strides(k, "k"), _head_strides(v, "v")
    gs = g.stride()
    shape = _b.mgs_attention_shape(B, 1, H, Hk, D, _DTYPES[dt], fixed, D ** -0.5 if scale is None else scale,
                                   (qb, 0, qh), (kb, 0, kh), (vb, 0, vh), (0, 0, 1) if fixed else (gs[0], 0, gs[1]))
    _b.mgs_linear_attention_step(shape, q, k, v, g, S, slots, S.shape[0], out, stream)
    _written(written)
    return out


# ---------------------------------------------------------------- RMS norm with the residual's addition
def _norm_args(x, weight, residual):
    try:  # the usual case in few steps: a call on one token takes less time on the GPU than its checks
        dt, shape, here = x.dtype, x.shape, x.get_device()
        N = shape[-1]
        if (dt in _DTYPES and here >= 0 and x.is_contiguous() and weight.dtype is dt and weight.shape == (N,)
                and weight.is_contiguous() and weight.get_device() == here
                and (residual is None or (residual.dtype is dt and residual.shape == shape
                                          and residual.is_contiguous() and residual.get_device() == here))):
            return x.numel() // N if N else shape[:-1].numel(), N, _DTYPES[dt]
    except (AttributeError, IndexError):
        pass
    _check_typed(x, "x", None, None)
    if x.dim() == 0:
        raise ValueError("x must have a last dimension")
    N = x.shape[-1]
    _check_typed(weight, "weight", (N,), x.dtype, device=x.device)
    if residual is not None:
        _check_typed(residual, "residual", x.shape, x.dtype, device=x.device)
    return x.numel() // N if N else x.shape[:-1].numel(), N, _DTYPES[x.dtype]


def rms_norm_fwd(x, weight, residual=None, eps=1e-6, stream=None):
    """r = x + residual (x itself without one), y = r weight / sqrt(mean(r^2) + eps) over the last dimension.
    x, residual [..., N], weight [N], all fp32 or all bf16.  Returns (y, r, rstd), rstd fp32 for the backward."""
    rows, N, dt = _norm_args(x, weight, residual)
    y = torch.empty_like(x)
    r = torch.empty_like(x) if residual is not None else None
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _b.mgs_rms_norm_fwd(x, residual, weight, eps, r, y, rstd, rows, N, dt, stream)
    return y, (r if r is not None else x), rstd


def rms_norm_fp8_fwd(x, weight, residual=None, eps=1e-6, group=0, stream=None):
    """The same with y in 8 bits (float8_e4m3fn) and fp32 scales: y = q * scale, a scale for each row (group 0) or
    each 128 columns of a row (group 128).  Returns (q, scales, r)."""
    rows, N, dt = _norm_args(x, weight, residual)
    if group not in (0, 128) or (group and N % group):
        raise ValueError("group must be 0, or 128 with a last dimension that it divides")
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    r = torch.empty_like(x) if residual is not None else None
    scales = torch.empty((*x.shape[:-1], N // group if group else 1), dtype=torch.float32, device=x.device)
    _b.mgs_rms_norm_fp8_fwd(x, residual, weight, eps, r, q, scales, rows, N, group, dt, stream)
    return q, scales, (r if r is not None else x)


def rms_norm_bwd(r, weight, rstd, grad_y, grad_r=None, stream=None):
    """Gradients of rms_norm_fwd: (dx, dweight); dx is that of x and of residual alike, grad_r (or None) what
    arrives at r itself."""
    rows, N, dt = _norm_args(r, weight, None)
    _check_typed(rstd, "rstd", r.shape[:-1], torch.float32, device=r.device)
    _check_typed(grad_y, "grad_y", r.shape, r.dtype, device=r.device)
    if grad_r is not None:
        _check_typed(grad_r, "grad_r", r.shape, r.dtype, device=r.device)
    dx, dw = torch.empty_like(r), torch.empty_like(weight)
    n = _b.mgs_rms_norm_bwd_workspace_size(rows, N)
    _b.mgs_rms_norm_bwd(r, weight, rstd, grad_y, grad_r, dx, dw, rows, N, dt, _scratch(n, r.device, stream), n, stream)
    return dx, dw


# ---------------------------------------------------------------- clipping by the global norm
def clip_grad_norm(grads, max_norm, out=None, stream=None):
    """The norm over all of grads (fp32 and bf16 tensors, contiguous) as one fp32 on the device, and the tensors
    scaled by min(1, max_norm / (norm + 1e-6)): in place, or into `out` (tensors of the same sizes and types).  No
    tensor is listed twice in place (tied parameters have one gradient), and no output lies over another tensor."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(outs)} outputs for {len(grads)} tensors")
    if not grads:
        raise ValueError("no tensors")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("each of grads must be a CUDA tensor (the library runs only on the GPU)")
    # whole lists at a time: there may be hundreds of tensors, and the check of each should cost little
    T, dtype = torch.Tensor, operator.attrgetter("dtype")
    here, n = [grads[0].get_device()] * len(grads), len(grads)
    types, sizes = list(map(dtype, grads)), list(map(T.numel, grads))
    codes = list(map(_DTYPES.get, types))
    if None in codes or list(map(T.get_device, grads)) != here or not all(map(T.is_contiguous, grads)):
        for t in grads:
            _check_typed(t, "each of grads", None, None, device=dev)
    to = at = list(map(T.data_ptr, grads))
    if out is not None:
        if (list(map(dtype, outs)) != types or list(map(T.numel, outs)) != sizes
                or list(map(T.get_device, outs)) != here or not all(map(T.is_contiguous, outs))):
            for t, u in zip(grads, outs):
                _check_typed(u, "each of out", t.shape, t.dtype, device=dev)
        to = list(map(T.data_ptr, outs))
    norm = torch.empty((), dtype=torch.float32, device=dev)
    size = _b.mgs_clip_grad_norm_workspace_size(n)
    _b.mgs_clip_grad_norm(at, to, sizes, codes, max_norm, norm, _scratch(size, dev, stream), size, stream)
    _written(outs)
    return norm


# ---------------------------------------------------------------- gated linear recurrence
def _elsewhere(t):
    """Whether t is on another GPU than the current one, on which the library would launch."""
    here = t.get_device()
    return here >= 0 and here != torch._C._cuda_getDevice()


def _inner(t, name):
    """Strides of all but the last dimension, which is contiguous."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return st[:-1]


def _gated_shape(gate, value, positive, grad_h=None):
    try:  # the usual case in few steps
        dt, shape, here, (kb, kt, kd), (vb, vt, vd) = gate.dtype, gate.shape, gate.get_device(), gate.stride(), value.stride()
        gb, gt, gd = (0, 0, 1) if grad_h is None else grad_h.stride()
        if (dt in _DTYPES and here >= 0 and value.dtype is dt and value.shape == shape and value.get_device() == here
                and kd == 1 and vd == 1 and gd == 1
                and (grad_h is None or grad_h.dtype is dt and grad_h.shape == shape and grad_h.get_device() == here)):
            return _b.mgs_gated_shape(*shape, _DTYPES[dt], bool(positive), (kb, kt), (vb, vt), (gb, gt))
    except (AttributeError, ValueError):
        pass
    if not isinstance(gate, torch.Tensor) or gate.dim() != 3:
        raise ValueError("gate must be a [B,T,D] tensor")
    _check_typed(gate, "gate", None, None, dense=False)
    _check_typed(value, "value", gate.shape, gate.dtype, dense=False, device=gate.device)
    if grad_h is not None:
        _check_typed(grad_h, "grad_h", gate.shape, gate.dtype, dense=False, device=gate.device)
    B, T, D = gate.shape
    return _b.mgs_gated_shape(B, T, D, _DTYPES[gate.dtype], bool(positive), _inner(gate, "gate"), _inner(value, "value"),
                              _inner(grad_h, "grad_h") if grad_h is not None else (0, 0))


def gated_scan_fwd(gate, value, h0=None, positive=True, want_carries=False, stream=None):
    """The gated linear recurrence (minGRU) from its pre-activations: with z = sigmoid(gate),
    h_t = (1 - z_t) h_{t-1} + z_t c_t, c = g(value) (positive: v + 1/2 for v >= 0, sigmoid(v) below) or value itself.

    gate, value [B,T,D] (fp32 or bf16, any strides whose channels are contiguous, so halves of one product too),
    h0 [B,D] fp32 or None.  A gate of -inf masks its step, whatever its value; +inf starts the state anew.  The
    state is fp32, h is rounded once.  Returns (h [B,T,D], h_T [B,D] fp32), and the carries that gated_scan_bwd
    takes when want_carries."""
    shape = _gated_shape(gate, value, positive)
    if _elsewhere(gate):
        with torch.cuda.device(gate.device):
            return gated_scan_fwd(gate, value, h0, positive, want_carries, stream)
    (B, T, D), dev = gate.shape, gate.device
    if h0 is not None:
        _check_typed(h0, "h0", (B, D), torch.float32, device=dev)
    h = torch.empty((B, T, D), dtype=gate.dtype, device=dev)
    hT = torch.empty((B, D), dtype=torch.float32, device=dev)
    carries = torch.empty((B, -(-T // _b.GATED_SPAN), D), dtype=torch.float32, device=dev) if want_carries else None
    _b.mgs_gated_scan_fwd(shape, gate, value, h0, h, hT, carries, stream)
    return (h, hT, carries) if want_carries else (h, hT)


def gated_scan_bwd(gate, value, carries, grad_h, grad_hT=None, positive=True, need_dh0=True, stream=None):
    """Gradients of gated_scan_fwd for L = <grad_h, h> + <grad_hT, h_T>: (dgate, dvalue, dh0), dh0 None unless
    needed.  carries: the forward's; h itself is rebuilt from them."""
    shape = _gated_shape(gate, value, positive, grad_h)
    if _elsewhere(gate):
        with torch.cuda.device(gate.device):
            return gated_scan_bwd(gate, value, carries, grad_h, grad_hT, positive, need_dh0, stream)
    (B, T, D), dev = gate.shape, gate.device
    _check_typed(carries, "carries", (B, -(-T // _b.GATED_SPAN), D), torch.float32, device=dev)
    if grad_hT is not None:
        _check_typed(grad_hT, "grad_hT", (B, D), torch.float32, device=dev)
    dgate = torch.empty((B, T, D), dtype=gate.dtype, device=dev)
    dvalue = torch.empty_like(dgate)
    dh0 = torch.empty((B, D), dtype=torch.float32, device=dev) if need_dh0 else None
    _b.mgs_gated_scan_bwd(shape, gate, value, carries, grad_h, grad_hT, dgate, dvalue, dh0, stream)
    return dgate, dvalue, dh0


def gated_scan_step(gate, value, state, slots=None, positive=True, out=None, stream=None):
    """One step of each of B sequences: gate, value [B,D], the cache of states [N,D] fp32, updated in place.
    slots [B] int32: each sequence's place in the cache (None: b itself); a place outside 0..N-1 marks an empty row,
    whose output is 0.  Returns h [B,D]."""
    try:  # the usual case in few steps: a call on one token takes less time on the GPU than its checks
        (B, D), dt, here, (kb, kd), (vb, vd), N = gate.shape, gate.dtype, gate.get_device(), gate.stride(), value.stride(), len(state)
        usual = (dt in _DTYPES and here >= 0 and value.dtype is dt and value.shape == gate.shape and value.get_device() == here
                 and kd == 1 and vd == 1 and state.dtype is torch.float32 and state.shape == (N, D)
                 and state.is_contiguous() and state.get_device() == here and out is None
                 and (N >= B if slots is None else slots.dtype is torch.int32 and slots.shape == (B,)
                      and slots.is_contiguous() and slots.get_device() == here))
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        B, D, N = _gated_step_check(gate, value, state, slots, out)
        dt, (kb, _), (vb, _) = gate.dtype, gate.stride(), value.stride()
    if _elsewhere(gate):
        with torch.cuda.device(gate.device):
            return gated_scan_step(gate, value, state, slots, positive, out, stream)
    written = (state,) if out is None else (state, out)
    if out is None:
        out = torch.empty((B, D), dtype=dt, device=gate.device)
    shape = _b.mgs_gated_shape(B, 1, D, _DTYPES[dt], bool(positive), (kb, 0), (vb, 0))
    _b.mgs_gated_scan_step(shape, gate, value, state, slots, N, out, stream)
    _written(written)
    return out


def _gated_step_check(gate, value, state, slots, out):
    if not isinstance(gate, torch.Tensor) or gate.dim() != 2:
        raise ValueError("gate must be a [B,D] tensor")
    (B, D), dt, dev = gate.shape, gate.dtype, gate.device
    _check_typed(gate, "gate", None, None, dense=False)
    _check_typed(value, "value", gate.shape, dt, dense=False, device=dev)
    _inner(gate, "gate"), _inner(value, "value")
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be a [N,D] tensor")
    N = state.shape[0]
    _check_typed(state, "state", (N, D), torch.float32, device=dev)
    if slots is not None:
        _check_typed(slots, "slots", (B,), torch.int32, device=dev)
    elif N < B:
        raise ValueError(f"{B} sequences without slots need a cache of as many states, not {N}")
    if out is not None:
        _check_typed(out, "out", (B, D), dt, device=dev)
    return B, D, N


# ---------------------------------------------------------------- norm of queries and keys, with the position's rotation
def rotary_table(positions, rotary, base=10000.0, device="cuda"):
    """The cosines and sines [positions, rotary] fp32 that qk_norm takes: of p base^(-2 i / rotary) for position p and
    pair i, computed in 64 bits (an angle of a far position in 32 bits is off by itself times 6e-8)."""
    if rotary % 2:
        raise ValueError("rotary must be even")
    i = torch.arange(rotary // 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * base ** (-2 * i / max(rotary, 1))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _qk_shape(q, k, q_weight, k_weight, table, positions, eps, interleaved, grad_q=None, grad_k=None):
    """The checked arguments as the C struct.  One token of each sequence ([B,H,D]) is T = 1."""
    try:  # the usual case in few steps
        qs, ks, dt, here, nd = q.shape, k.shape, q.dtype, q.get_device(), len(q.shape)
        D, one = qs[-1], nd == 3
        usual = (dt in _DTYPES and here >= 0 and k.dtype is dt and k.get_device() == here and 3 <= nd <= 4 and len(ks) == nd
                 and qs[0] == ks[0] and (one or qs[1] == ks[1]) and ks[-1] == D and D % 8 == 0 and 8 <= D <= 256)
        for w in (q_weight, k_weight):
            usual = usual and (w is None or w.dtype is dt and w.shape == (D,) and w.get_device() == here and w.is_contiguous())
        rows, R = 0, 0
        if table is not None:
            rows, R = table.shape
            usual = (usual and table.dtype is torch.float32 and table.is_contiguous() and table.get_device() == here
                     and R % 8 == 0 and 8 <= R <= D and (positions is not None or rows >= (1 if one else qs[1])))
        at = (0, 0)
        if positions is not None:
            usual = (usual and table is not None and positions.dtype is torch.int32 and positions.shape == qs[:-2]
                     and positions.get_device() == here)
            at = (positions.stride(0), 0) if one else positions.stride()
        none = (0, 0, 0)
        strides = [none if t is None else t.stride() for t in (q, k, grad_q, grad_k)]
        for t, like, st in ((q, q, strides[0]), (k, k, strides[1]), (grad_q, q, strides[2]), (grad_k, k, strides[3])):
            usual = usual and (t is None or st[-1] == 1 and (t is like or t.dtype is dt and t.shape == like.shape
                                                            and t.get_device() == here))
    except (AttributeError, IndexError, TypeError, ValueError):
        usual = False
    if not usual:
        return _qk_shape_checked(q, k, q_weight, k_weight, table, positions, eps, interleaved, grad_q, grad_k)
    strides = [st if st is none else (st[0], 0, st[1]) if one else st[:3] for st in strides]
    return _b.mgs_qk_norm_shape(qs[0], 1 if one else qs[1], qs[-2], ks[-2], rows, D, _DTYPES[dt], R, bool(interleaved), eps,
                                *strides, at)


def _qk_shape_checked(q, k, q_weight, k_weight, table, positions, eps, interleaved, grad_q, grad_k):
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise ValueError("q must be a [B,T,Hq,D] or [B,Hq,D] tensor")
    dt, dev, D, lead = q.dtype, q.device, q.shape[-1], q.shape[:-2]
    _check_typed(q, "q", None, None, dense=False)
    if not isinstance(k, torch.Tensor) or k.dim() != q.dim():
        raise ValueError("k must have as many dimensions as q")
    _check_typed(k, "k", (*lead, k.shape[-2], D), dt, dense=False, device=dev)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _check_typed(w, name, (D,), dt, device=dev)
    if D % 8 or not 8 <= D <= 256:
        raise ValueError(f"heads of {D}: multiples of 8 up to 256 are supported")
    rows, R = 0, 0
    if table is not None:
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("table must be a [positions, rotary] tensor")
        rows, R = table.shape
        _check_typed(table, "table", None, torch.float32, device=dev)
        if R % 8 or not 8 <= R <= D:
            raise ValueError(f"{R} rotated elements of heads of {D}: multiples of 8 up to {D} are supported")
        if positions is None and rows < (lead[1] if len(lead) == 2 else 1):
            raise ValueError(f"{lead[1] if len(lead) == 2 else 1} positions need a table of as many rows, not {rows}")
    if positions is not None:
        if table is None:
            raise ValueError("positions without a table")
        _check_typed(positions, "positions", lead, torch.int32, dense=False, device=dev)
    for g, like, name in ((grad_q, q, "grad_q"), (grad_k, k, "grad_k")):
        if g is not None:
            _check_typed(g, name, like.shape, dt, dense=False, device=dev)
    one = len(lead) == 1

    def strides(t, name):
        st = _inner(t, name) if t is not None else (0,) * (len(lead) + 1)
        return (st[0], 0, st[1]) if one else st

    at = (0, 0) if positions is None else (*positions.stride(), 0) if one else positions.stride()
    return _b.mgs_qk_norm_shape(lead[0], 1 if one else lead[1], q.shape[-2], k.shape[-2], rows, D, _DTYPES[dt], R,
                                bool(interleaved), eps, strides(q, "q"), strides(k, "k"), strides(grad_q, "grad_q"),
                                strides(grad_k, "grad_k"), at)


def qk_norm_fwd(q, k, q_weight=None, k_weight=None, table=None, positions=None, eps=1e-6, interleaved=False, stream=None):
    """RMS norm of queries and keys over each head's D elements, times the weights [D] (None: ones), then the rotation
    of their positions, in one pass: what linear_attention takes.

    q [B,T,Hq,D], k [B,T,Hk,D], or [B,H,D] for one token of each sequence (fp32 or bf16, D a multiple of 8 up to 256, any
    strides whose heads are contiguous).  table: rotary_table's, as many elements of a head turned as it has columns
    (None: none); pairs are elements i and i + rotary / 2, or 2 i and 2 i + 1 (interleaved).  positions [B,T] or [B]
    int32 (None: 0..T-1); one outside the table marks an empty row, whose outputs and gradients are 0.  Sums and
    rotations are fp32, outputs are rounded once.  Returns dense (q, k)."""
    shape = _qk_shape(q, k, q_weight, k_weight, table, positions, eps, interleaved)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return qk_norm_fwd(q, k, q_weight, k_weight, table, positions, eps, interleaved, stream)
    yq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    yk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    _b.mgs_qk_norm_fwd(shape, q, k, q_weight, k_weight, table, positions, yq, yk, stream)
    return yq, yk


def qk_norm_bwd(q, k, q_weight, k_weight, grad_q, grad_k, table=None, positions=None, eps=1e-6, interleaved=False,
                stream=None):
    """Gradients of qk_norm_fwd: (dq, dk, dq_weight, dk_weight), those of weights that are None None."""
    if grad_q is None or grad_k is None:
        raise ValueError("grad_q and grad_k must be tensors")
    shape = _qk_shape(q, k, q_weight, k_weight, table, positions, eps, interleaved, grad_q, grad_k)
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return qk_norm_bwd(q, k, q_weight, k_weight, grad_q, grad_k, table, positions, eps, interleaved, stream)
    dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    dqw, dkw = (None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
    n = _b.mgs_qk_norm_bwd_workspace_size(shape)
    _b.mgs_qk_norm_bwd(shape, q, k, q_weight, k_weight, grad_q, grad_k, table, positions, dq, dk, dqw, dkw,
                       _scratch(n, q.device, stream), n, stream)
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- embedding
_TOKENS = {torch.int32: _b.MGS_I32, torch.int64: _b.MGS_I64}


def _check_tokens(tokens, device=None):
    if not isinstance(tokens, torch.Tensor) or tokens.dtype not in _TOKENS:
        raise ValueError("tokens must be an int32 or int64 tensor")
    _check_typed(tokens, "tokens", None, tokens.dtype, device=device)


def embedding_fwd(tokens, weight, scale=1.0, stream=None):
    """scale * weight[tokens]: tokens [...] int32 or int64, weight [V,D] fp32 or bf16.  A token outside 0..V-1 marks an
    empty row, which is 0.  Returns [..., D]."""
    _check_typed(weight, "weight", None, None)
    if weight.dim() != 2:
        raise ValueError("weight must be a [V,D] tensor")
    _check_tokens(tokens, weight.device)
    if _elsewhere(weight):
        with torch.cuda.device(weight.device):
            return embedding_fwd(tokens, weight, scale, stream)
    V, D = weight.shape
    out = torch.empty((*tokens.shape, D), dtype=weight.dtype, device=weight.device)
    _b.mgs_embedding_fwd(tokens, _TOKENS[tokens.dtype], weight, scale, out, tokens.numel(), V, D, _DTYPES[weight.dtype],
                         stream)
    return out


def embedding_bwd(tokens, grad, V, scale=1.0, stream=None):
    """The gradient [V,D] of embedding_fwd's weight, dense: scale times the sum of grad's rows over each token's places
    (fp32 sums, in an order that the tokens alone decide).  grad [..., D]: rows a fixed distance apart."""
    _check_typed(grad, "grad", None, None, dense=False)
    _check_tokens(tokens, grad.device)
    if grad.dim() != tokens.dim() + 1 or grad.shape[:-1] != tokens.shape:
        raise ValueError(f"grad has shape {tuple(grad.shape)}, expected {(*tokens.shape, 'D')}")
    N, D = tokens.numel(), grad.shape[-1]
    try:
        rows = grad if grad.dim() == 2 else grad.view(N, D)
    except RuntimeError:
        raise ValueError("grad must have rows a fixed distance apart") from None
    apart, = _inner(rows, "grad")
    if _elsewhere(grad):
        with torch.cuda.device(grad.device):
            return embedding_bwd(tokens, grad, V, scale, stream)
    dW = torch.empty((V, D), dtype=grad.dtype, device=grad.device)
    n = _b.mgs_embedding_bwd_workspace_size(N, V, D)
    _b.mgs_embedding_bwd(tokens, _TOKENS[tokens.dtype], rows, apart, scale, dW, N, V, D, _DTYPES[grad.dtype],
                         _scratch(n, grad.device, stream), n, stream)
    return dW


# ---------------------------------------------------------------- autograd wrappers
class MatrixAffineScan(torch.autograd.Function):
    """h = matrix_affine_scan(A, b, h0) with the library's fused backward;
    recompute=True saves b instead of h and the backward rebuilds h."""

    @staticmethod
    def forward(ctx, A, b, h0=None, recompute=False):
        A, b = A.contiguous(), b.contiguous()
        h0c = h0.contiguous() if h0 is not None else None
        h = matrix_affine_scan_fwd(A, b, h0c)
        ctx.save_for_backward(A, h0c if h0c is not None else torch.empty(0, device=b.device), b if recompute else h)
        ctx.has_h0 = h0 is not None
        ctx.recompute = recompute
        return h

    @staticmethod
    def backward(ctx, grad_h):
        A, h0, x = ctx.saved_tensors
        h0 = h0 if ctx.has_h0 else None
        if ctx.recompute:
            dA, db, dh0 = matrix_affine_scan_bwd_recompute(A, x, h0, grad_h.contiguous(), need_dh0=ctx.has_h0)
        else:
            dA, db, dh0 = matrix_affine_scan_bwd(A, h0, x, grad_h.contiguous(), need_dh0=ctx.has_h0)
        return dA, db, dh0, None


class MatrixScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A):
        A = A.contiguous()
        P = matrix_scan_fwd(A)
        ctx.save_for_backward(A, P)
        return P

    @staticmethod
    def backward(ctx, grad_P):
        A, P = ctx.saved_tensors
        return matrix_scan_bwd(A, P, grad_P.contiguous())


class ParallelScanLog(torch.autograd.Function):
    @staticmethod
    def forward(ctx, log_coeffs, log_values, log_h0=None, recompute=False):
        lc, lv = log_coeffs.contiguous(), log_values.contiguous()
        l0 = log_h0.contiguous() if log_h0 is not None else None
        h = parallel_scan_log_fwd(lc, lv, l0)
        empty = torch.empty(0, device=lc.device)
        ctx.save_for_backward(lc, lv, l0 if l0 is not None else empty, empty if recompute else h)
        ctx.has_h0 = log_h0 is not None
        ctx.recompute = recompute
        return h

    @staticmethod
    def backward(ctx, grad_h):
        lc, lv, l0, h = ctx.saved_tensors
        l0 = l0 if ctx.has_h0 else None
        h = None if ctx.recompute else h
        dlc, dlv, dl0 = parallel_scan_log_bwd(lc, lv, l0, h, grad_h.contiguous())
        return dlc, dlv, dl0, None


class LinearScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, h0=None):
        a, b = a.contiguous(), b.contiguous()
        h0c = h0.contiguous() if h0 is not None else None
        h = linear_scan_fwd(a, b, h0c)
        ctx.save_for_backward(a, h0c if h0c is not None else torch.empty(0, device=a.device), h)
        ctx.has_h0 = h0 is not None
        return h

    @staticmethod
    def backward(ctx, grad_h):
        a, h0, h = ctx.saved_tensors
        h0 = h0 if ctx.has_h0 else None
        da, db, dh0 = linear_scan_bwd(a, h0, h, grad_h.contiguous(), need_dh0=ctx.has_h0)
        return da, db, dh0


class GivensAffineScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, theta, a, b, h0=None):
        theta, b = theta.contiguous(), b.contiguous()
        a = a.contiguous() if a is not None else None
        h0c = h0.contiguous() if h0 is not None else None
        h = givens_affine_scan_fwd(theta, a, b, h0c)
        empty = torch.empty(0, device=b.device)
        ctx.save_for_backward(theta, a if a is not None else empty, h0c if h0c is not None else empty, h)
        ctx.has_a, ctx.has_h0 = a is not None, h0 is not None
        return h

    @staticmethod
    def backward(ctx, grad_h):
        theta, a, h0, h = ctx.saved_tensors
        a = a if ctx.has_a else None
        h0 = h0 if ctx.has_h0 else None
        dth, da, db, dh0 = givens_affine_scan_bwd(theta, a, h0, h, grad_h.contiguous(), need_dh0=ctx.has_h0)
        return dth, da, db, dh0


class GivensMatrixScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, theta):
        theta = theta.contiguous()
        P = givens_matrix_scan_fwd(theta)
        ctx.save_for_backward(theta, P)
        return P

    @staticmethod
    def backward(ctx, grad_P):
        theta, P = ctx.saved_tensors
        return givens_matrix_scan_bwd(theta, P, grad_P.contiguous())


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, S0=None, scale=None):
        S0 = S0.contiguous() if S0 is not None else None
        o, ST = linear_attention_fwd(q, k, v, g, S0, scale, want_state=True)
        ctx.save_for_backward(q, k, v, g, S0)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, ST

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_o, grad_ST):
        q, k, v, g, S0 = ctx.saved_tensors
        if grad_o is None:
            grad_o = torch.zeros(v.shape, dtype=v.dtype, device=v.device)
        if grad_ST is not None:
            grad_ST = grad_ST.contiguous()
        dq, dk, dv, dg, dS0 = linear_attention_bwd(q, k, v, g, _aligned(grad_o), S0, grad_ST, ctx.scale)
        return dq, dk, dv, dg, dS0, None


class RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual=None, eps=1e-6):
        y, r, rstd = rms_norm_fwd(x.contiguous(), weight, residual.contiguous() if residual is not None else None, eps)
        ctx.save_for_backward(r, weight, rstd)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return (y, r) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_r=None):
        r, weight, rstd = ctx.saved_tensors
        grad_y = torch.zeros_like(r) if grad_y is None else grad_y.contiguous()
        dx, dw = rms_norm_bwd(r, weight, rstd, grad_y, grad_r.contiguous() if grad_r is not None else None)
        return dx, dw, dx if ctx.has_residual else None, None


def _dense_inner(t):
    """t itself where its last dimension is contiguous (or it is refused further on), else a dense copy."""
    return t.contiguous() if isinstance(t, torch.Tensor) and t.dim() and t.stride(-1) != 1 else t


def _zeros_like_rows(t):
    """Zeros of t's shape, one row of them in memory."""
    return torch.zeros(t.shape[-1], dtype=t.dtype, device=t.device).expand(t.shape)


class GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, value, h0=None, positive=True):
        h0 = h0.contiguous() if h0 is not None else None
        h, hT, carries = gated_scan_fwd(gate, value, h0, positive, want_carries=True)
        ctx.save_for_backward(gate, value, carries)
        ctx.positive, ctx.has_h0 = positive, h0 is not None
        ctx.set_materialize_grads(False)
        return h, hT

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h, grad_hT):
        gate, value, carries = ctx.saved_tensors
        grad_h = _zeros_like_rows(gate) if grad_h is None else _dense_inner(grad_h)
        grad_hT = grad_hT.contiguous() if grad_hT is not None else None
        dgate, dvalue, dh0 = gated_scan_bwd(gate, value, carries, grad_h, grad_hT, ctx.positive, ctx.has_h0)
        return dgate, dvalue, dh0, None


class QKNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        ctx.set_materialize_grads(False)
        return qk_norm_fwd(q, k, q_weight, k_weight, table, positions, eps, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_q, grad_k):
        q, k, q_weight, k_weight, table, positions = ctx.saved_tensors
        grad_q, grad_k = (_zeros_like_rows(x) if g is None else _dense_inner(g) for g, x in ((grad_q, q), (grad_k, k)))
        grads = qk_norm_bwd(q, k, q_weight, k_weight, grad_q, grad_k, table, positions, ctx.eps, ctx.interleaved)
        return *grads, None, None, None, None


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale=1.0):
        tokens = tokens.contiguous() if isinstance(tokens, torch.Tensor) else tokens
        out = embedding_fwd(tokens, weight, scale)
        ctx.save_for_backward(tokens)
        ctx.V, ctx.scale = weight.shape[0], scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        tokens, = ctx.saved_tensors
        return None, embedding_bwd(tokens, grad.contiguous(), ctx.V, ctx.scale), None


def givens_affine_scan(theta, a, b, h0=None):
    """GivensMinGRU's angle-fused recurrence h_t = G(theta_t) diag(a_t) h_{t-1} + b_t (a may be None)."""
    return GivensAffineScan.apply(theta, a, b, h0)


def givens_matrix_scan(theta):
    return GivensMatrixScan.apply(theta)


def linear_scan(a, b, h0=None):
    return LinearScan.apply(a, b, h0)


def matrix_affine_scan(A, b, h0=None, recompute=False):
    """recompute=True keeps b rather than h for backward; backward rebuilds h."""
    return MatrixAffineScan.apply(A, b, h0, recompute)


def matrix_scan(A):
    return MatrixScan.apply(A)


def parallel_scan_log(log_coeffs, log_values, log_h0=None, recompute=False):
    """recompute=True keeps no copy of h for backward; backward rebuilds it."""
    return ParallelScanLog.apply(log_coeffs, log_values, log_h0, recompute)


def _aligned(t):
    """t itself where its strides are ones the attention kernels take, else a dense copy."""
    es = t.element_size()
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s * es % 16 == 0 for s in t.stride()[:-1])
    return t if ok else t.contiguous()


def linear_attention(q, k, v, g, S0=None, scale=None):
    """Linear attention with a decay for each head, with gradients: (o, S_T); see linear_attention_fwd."""
    return LinearAttention.apply(_aligned(q), _aligned(k), _aligned(v), g, S0, scale)


def rms_norm(x, weight, residual=None, eps=1e-6):
    """RMS norm over the last dimension, with gradients: y, or (y, r) with r = x + residual."""
    return RMSNorm.apply(x, weight, residual, eps)


def gated_scan(gate, value, h0=None, positive=True):
    """The gated linear recurrence (minGRU) from its pre-activations, with gradients: (h, h_T); see gated_scan_fwd."""
    return GatedScan.apply(_dense_inner(gate), _dense_inner(value), h0, positive)


def qk_norm(q, k, q_weight=None, k_weight=None, table=None, positions=None, eps=1e-6, interleaved=False):
    """Norm of queries and keys for each head with their positions' rotation, with gradients: (q, k); see qk_norm_fwd."""
    return QKNorm.apply(_dense_inner(q), _dense_inner(k), q_weight, k_weight, table, positions, eps, interleaved)


def embedding(tokens, weight, scale=1.0):
    """scale * weight[tokens], with the gradient of weight; see embedding_fwd."""
    return Embedding.apply(tokens, weight, scale)
