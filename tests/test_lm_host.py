"""Checks of the language-model operators that need no GPU: the references of
their tests against differences, and the refusals of the C ABI (fake,
never-dereferenced addresses) and of the tensor-level functions."""
import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api
from scan_linear_recurrences_gb300.build import build

from . import _lm

FAKE = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = b.MGS_ERR_INVALID_ARG, b.MGS_ERR_UNSUPPORTED, b.MGS_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def _st(fn, *args):
    try:
        fn(*args, stream=0)
        return b.MGS_OK
    except b.MGSError as e:
        return e.status


def test_attention_reference_gradients_against_differences():
    d = _lm.attn_inputs(2, 5, 4, 2, 3, seed=3)
    ref = _lm.attn_ref(d)
    gen = torch.Generator().manual_seed(4)

    def loss(x):
        o, ST = _lm.attn_forward64(x["q"], x["k"], x["v"], x["g"], x["S0"], 3 ** -0.5)
        return (o * d["grad_o"].double()).sum() + (ST * d["grad_ST"].double()).sum()

    # central differences in 64 bits: truncation eps^2, rounding 1e-16 / eps
    for n in ("q", "k", "v", "g", "S0"):
        x = {m: d[m].double() for m in ("q", "k", "v", "g", "S0")}
        u = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        hi, lo = loss({**x, n: x[n] + eps * u}), loss({**x, n: x[n] - eps * u})
        want = (ref["d" + n] * u).sum()
        assert abs((hi - lo) / (2 * eps) - want) <= 1e-7 * (1 + abs(want)), n


def test_norm_reference_gradients_against_differences():
    gen = torch.Generator().manual_seed(5)
    x, res, w, gy, gr = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 7), (3, 7), (7,), (3, 7), (3, 7)))

    def loss(x, w):
        o = _lm.norm_ref(x, w, None, 1e-6, torch.float64)
        return (o["y"] * gy).sum() + (o["r"] * gr).sum()

    ref = _lm.norm_ref(x, w, None, 1e-6, torch.float64, gy, gr)
    u, uw, eps = torch.randn_like(x), torch.randn_like(w), 1e-5
    for hi, lo, want in ((loss(x + eps * u, w), loss(x - eps * u, w), (ref["dx"] * u).sum()),
                         (loss(x, w + eps * uw), loss(x, w - eps * uw), (ref["dw"] * uw).sum())):
        assert abs((hi - lo) / (2 * eps) - want) <= 1e-7 * (1 + abs(want))


def _shape(B=2, T=8, H=4, Hk=2, D=64, dtype=b.MGS_BF16, fixed=0, qs=None, gs=None):
    s = (T * Hk * D, Hk * D, D)
    v = (T * H * D, H * D, D)
    return b.mgs_attention_shape(B, T, H, Hk, D, dtype, fixed, 0.125, qs or s, s, v, gs or (T * H, H, 1), v)


def test_attention_refusals():
    q, k, v, g, S0, o, ST = (FAKE + i * (1 << 30) for i in range(7))
    ws = FAKE + (7 << 30)
    f = b.mgs_linear_attention_fwd
    assert _st(f, None, q, k, v, g, S0, o, ST) == INVALID
    assert _st(f, _shape(B=-1), q, k, v, g, S0, o, ST) == INVALID
    assert _st(f, _shape(H=4, Hk=3), q, k, v, g, S0, o, ST) == INVALID       # 3 does not divide 4
    assert _st(f, _shape(H=4, Hk=0), q, k, v, g, S0, o, ST) == INVALID
    assert _st(f, _shape(D=96), q, k, v, g, S0, o, ST) == UNSUPPORTED
    assert _st(f, _shape(dtype=7), q, k, v, g, S0, o, ST) == UNSUPPORTED
    assert _st(f, _shape(qs=(1024, 132, 64)), q, k, v, g, S0, o, ST) == UNSUPPORTED   # 264 bytes
    assert _st(f, _shape(qs=(-1024, 128, 64)), q, k, v, g, S0, o, ST) == UNSUPPORTED
    assert _st(f, _shape(), q + 8, k, v, g, S0, o, ST) == UNSUPPORTED
    assert _st(f, _shape(), q, k, v, g + 2, S0, o, ST) == UNSUPPORTED
    assert _st(f, _shape(), q, None, v, g, S0, o, ST) == INVALID
    assert _st(f, _shape(), q, k, v, None, S0, o, ST) == INVALID
    assert _st(f, _shape(B=1 << 31, T=1 << 31), q, k, v, g, S0, o, ST) == INVALID
    assert _st(f, _shape(B=0), None, None, None, None, None, None, None) == b.MGS_OK
    # outputs over inputs, or over each other
    n = b.mgs_linear_attention_workspace_size(_shape(), 0)
    assert _st(f, _shape(), q, k, v, g, S0, v + 64, ST, ws, n) == INVALID
    assert _st(f, _shape(), q, k, v, g, S0, o, S0, ws, n) == INVALID
    assert _st(f, _shape(), q, k, v, g, S0, o, o, ws, n) == INVALID


def test_attention_workspace():
    # few lanes and long: segments; its size does not depend on the strides
    long = _shape(B=1, T=8192, H=2, Hk=2, D=128)
    n = b.mgs_linear_attention_workspace_size(long, 0)
    assert n > 0
    q, k, v, g, S0, o, ST, ws = (FAKE + i * (1 << 34) for i in range(8))
    f = b.mgs_linear_attention_fwd
    assert _st(f, long, q, k, v, g, S0, o, ST) == WORKSPACE
    assert _st(f, long, q, k, v, g, S0, o, ST, ws, n - 1) == WORKSPACE
    assert _st(f, long, q, k, v, g, S0, o, ST, ws + 16, n) == WORKSPACE
    assert _st(f, long, q, k, v, g, S0, o, ST, q, n) == INVALID
    assert b.mgs_linear_attention_workspace_size(_shape(D=96), 1) == 0
    bwd = b.mgs_linear_attention_bwd
    outs = [FAKE + (i << 34) for i in range(8, 13)]
    assert _st(bwd, _shape(), q, k, v, g, S0, o, ST, *outs) == WORKSPACE
    assert _st(bwd, _shape(), q, k, v, g, S0, None, ST, *outs) == INVALID
    n = b.mgs_linear_attention_workspace_size(_shape(), 1)
    assert _st(bwd, _shape(), q, k, v, g, S0, o, ST, outs[0], outs[0], *outs[2:], ws, n) == INVALID


def test_step_refusals():
    q, k, v, g, S, slots, o = (FAKE + i * (1 << 30) for i in range(7))
    f = b.mgs_linear_attention_step
    assert _st(f, _shape(T=2), q, k, v, g, S, slots, 8, o) == INVALID
    assert _st(f, _shape(T=1), q, k, v, g, S, None, 1, o) == INVALID         # fewer states than sequences
    assert _st(f, _shape(T=1), q, k, v, g, S, slots, -1, o) == INVALID
    assert _st(f, _shape(T=1), q, k, v, g, S, slots + 2, 8, o) == UNSUPPORTED
    assert _st(f, _shape(T=1), q, k, v, g, S, slots, 8, S) == INVALID
    assert _st(f, _shape(T=1, B=0), None, None, None, None, None, None, 0, None) == b.MGS_OK


def test_norm_refusals():
    x, res, w, r, y, rstd = (FAKE + i * (1 << 30) for i in range(6))
    f, f8, bwd = b.mgs_rms_norm_fwd, b.mgs_rms_norm_fp8_fwd, b.mgs_rms_norm_bwd
    assert _st(f, x, res, w, 1e-6, None, y, rstd, 4, 64, b.MGS_F32) == INVALID    # a residual without r
    assert _st(f, x, None, w, 1e-6, r, y, rstd, 4, 64, b.MGS_F32) == INVALID
    assert _st(f, x, res, w, 1e-6, r, y, rstd, -1, 64, b.MGS_F32) == INVALID
    assert _st(f, x, res, w, 1e-6, r, y, rstd, 4, 64, 9) == UNSUPPORTED
    assert _st(f, x + 1, res, w, 1e-6, r, y, rstd, 4, 64, b.MGS_BF16) == UNSUPPORTED
    assert _st(f, x, res, w, 1e-6, r, x, rstd, 4, 64, b.MGS_F32) == INVALID
    assert _st(f, None, None, None, 1e-6, None, None, None, 0, 64, b.MGS_F32) == b.MGS_OK
    assert _st(f8, x, res, w, 1e-6, r, y, rstd, 4, 64, 128, b.MGS_F32) == UNSUPPORTED
    assert _st(f8, x, res, w, 1e-6, r, y, rstd, 4, 256, 64, b.MGS_F32) == UNSUPPORTED
    assert _st(f8, x, res, w, 1e-6, r, y, None, 4, 256, 128, b.MGS_F32) == INVALID
    n = b.mgs_rms_norm_bwd_workspace_size(4, 64)
    assert n >= 4 * 64
    assert _st(bwd, r, w, rstd, y, None, x, res, 4, 64, b.MGS_F32) == WORKSPACE
    assert _st(bwd, r, w, None, y, None, x, res, 4, 64, b.MGS_F32, FAKE + (9 << 30), n) == INVALID
    assert _st(bwd, r, w, rstd, y, None, y, res, 4, 64, b.MGS_F32, FAKE + (9 << 30), n) == INVALID


def test_clip_refusals():
    f = lambda *a: _st(b.mgs_clip_grad_norm, *a)  # noqa: E731
    a, c, norm, ws = (FAKE + i * (1 << 30) for i in range(4))
    n = b.mgs_clip_grad_norm_workspace_size(1)
    assert f([a], [a], [8], [b.MGS_F32], -1.0, norm, ws, n) == INVALID
    assert f([a], [a], [8], [b.MGS_F32], float("nan"), norm, ws, n) == INVALID
    assert f([a], [a], [8], [5], 1.0, norm, ws, n) == UNSUPPORTED
    assert f([a + 2], [a + 2], [8], [b.MGS_F32], 1.0, norm, ws, n) == UNSUPPORTED
    assert f([a], [a + 16], [8], [b.MGS_F32], 1.0, norm, ws, n) == INVALID     # neither in place nor apart
    assert f([a], [a], [8], [b.MGS_F32], 1.0, a, ws, n) == INVALID             # the norm inside a tensor
    assert f([a], [a], [8], [b.MGS_F32], 1.0, None, ws, n) == INVALID
    assert f([a], [a], [-8], [b.MGS_F32], 1.0, norm, ws, n) == INVALID
    assert f([a], [a], [8], [b.MGS_F32], 1.0, norm, None, 0) == WORKSPACE
    assert f([None or 0], [0], [8], [b.MGS_F32], 1.0, norm, ws, n) == INVALID


def test_tensor_functions_refuse_cpu_tensors_and_wrong_types():
    d = _lm.attn_inputs(1, 4, 2, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_attention_fwd(d["q"], d["k"], d["v"], d["g"])
    with pytest.raises(ValueError, match=r"\[B,T,Hk,D\]"):
        api.linear_attention_fwd(d["q"][0], d["k"], d["v"], d["g"])
    with pytest.raises(ValueError, match="CUDA"):
        api.rms_norm_fwd(torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        api.clip_grad_norm([torch.zeros(8)], 1.0)
    with pytest.raises(ValueError, match="no tensors"):
        api.clip_grad_norm([], 1.0)
