"""GPU parity of the language-model operators against 64-bit references:
linear attention with a decay for each head (forward, gradients, single
tokens), the RMS norm with the residual's addition (and its fp8 output), and
clipping by the global norm; the lengths, head layouts, strides, decays and
special values at which each can go wrong."""
import math

import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api
from scan_linear_recurrences_gb300.build import build

from . import _lm
from ._lm import BF16_ONE, BF16_TWO, FP32, check, check_rounded

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    build()
    b.lib()
    yield
    b.mgs_check()


def _run_attn(d, scale=None, grads=True):
    c = _lm.cuda(d)
    o, ST = api.linear_attention_fwd(c["q"], c["k"], c["v"], c["g"], c["S0"], scale, want_state=True)
    out = {"o": o, "S_T": ST}
    if grads:
        r = api.linear_attention_bwd(c["q"], c["k"], c["v"], c["g"], c["grad_o"], c["S0"], c["grad_ST"], scale)
        out.update(zip(("dq", "dk", "dv", "dg", "dS0"), r))
    b.mgs_check()
    return out


def _compare(got, ref, dtype):
    tol = FP32 if dtype == F32 else BF16_TWO
    for n, r in ref.items():
        check(n, got[n], r, FP32 if n in ("S_T", "dg", "dS0") else tol)


# ---------------------------------------------------------------- linear attention
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,H,Hk,D,S0,fixed", [
    (1, 1, 1, 1, 64, True, False), (2, 1, 2, 1, 128, False, True), (1, 2, 3, 3, 64, False, False),
    (2, 15, 2, 2, 128, True, False), (1, 17, 5, 5, 64, True, True), (3, 63, 2, 2, 64, True, False),
    (1, 127, 2, 1, 128, True, False), (2, 128, 2, 2, 128, False, False), (1, 129, 3, 1, 64, True, False),
    (1, 200, 6, 2, 64, True, True), (2, 257, 4, 4, 128, True, False), (1, 300, 3, 3, 128, False, True),
    (3, 383, 2, 1, 128, True, False),
])
def test_attention_shapes(B, T, H, Hk, D, S0, fixed, dtype):
    d = _lm.attn_inputs(B, T, H, Hk, D, dtype, S0, fixed, seed=B * 1000 + T + H)
    _compare(_run_attn(d), _lm.attn_ref(d), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,H,Hk,D,S0", [
    (1, 1024, 1, 1, 128, True), (1, 1025, 2, 1, 64, True), (1, 2500, 1, 1, 64, False), (2, 1300, 3, 3, 64, True),
    (1, 2177, 2, 2, 128, False),
])
def test_attention_segments_and_spans(B, T, H, Hk, D, S0, dtype):
    # few lanes: time cut into segments; past 1024 steps: several spans of the decay's gradient
    d = _lm.attn_inputs(B, T, H, Hk, D, dtype, S0, seed=T, decay=0.05)
    _compare(_run_attn(d), _lm.attn_ref(d), dtype)


@pytest.mark.parametrize("D,dtype", [(64, F32), (64, BF16), (128, BF16), (128, F32)])
def test_attention_many_lanes(D, dtype):
    # more lanes than SMs: every lane one walk; an odd number of heads
    d = _lm.attn_inputs(53, 140, 3, 3, D, dtype, False, seed=9)
    _compare(_run_attn(d), _lm.attn_ref(d), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_strided_inputs(D, dtype):
    # q, k, v as parts of one projection, and as [B,H,T,D]; g as [B,H,T]; grad_o a broadcast
    B, T, H = 2, 150, 2
    gen = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, T, 3 * H * D, generator=gen).to(dtype).cuda()
    q, k, v = (qkv[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    g = (-torch.rand(B, H, T, generator=gen)).cuda().transpose(1, 2)
    go = torch.randn(1, 1, H, D, generator=gen).to(dtype).cuda().expand(B, T, H, D)
    want = api.linear_attention_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous())
    assert torch.equal(api.linear_attention_fwd(q, k, v, g), want)
    qt, kt, vt = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v))
    assert torch.equal(api.linear_attention_fwd(qt, kt, vt, g), want)
    got = api.linear_attention_bwd(q, k, vt, g, go)
    dense = api.linear_attention_bwd(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), go.contiguous())
    for x, y in zip(got[:4], dense[:4]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_zero_strides_through_the_c_entry(dtype):
    # keys broadcast over the steps: no tensor map has a zero stride, so the
    # entry point takes the kernel that needs none
    d = _lm.attn_inputs(2, 60, 2, 2, 64, dtype, False, seed=12)
    d["k"] = d["k"][:, :1].expand(2, 60, 2, 64)
    c = _lm.cuda(d)
    k = c["k"][:, :1].contiguous()
    dense = (60 * 128, 128, 64)
    shape = b.mgs_attention_shape(2, 60, 2, 2, 64, b.MGS_F32 if dtype == F32 else b.MGS_BF16, 0, 0.125, dense,
                                  (128, 0, 64), dense, (120, 2, 1))
    n = b.mgs_linear_attention_workspace_size(shape, 0)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    o = torch.empty(2, 60, 2, 64, dtype=dtype, device="cuda")
    ST = torch.empty(2, 2, 64, 64, device="cuda")
    b.mgs_linear_attention_fwd(shape, c["q"], k, c["v"], c["g"], None, o, ST, ws, n)
    b.mgs_check()
    _compare({"o": o, "S_T": ST}, _lm.attn_ref(d, grads=False), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_reset_and_strong_decays(dtype):
    # a decay of zero (g = -inf) starts the state anew: the steps before do not
    # reach those after; very strong and vanishing decays in one sequence
    B, T, H, D = 1, 300, 2, 64
    d = _lm.attn_inputs(B, T, H, H, D, dtype, True, seed=21)
    for t in (0, 37, 128, 200, 255):
        d["g"][:, t, 0] = -math.inf
    d["g"][:, 50:60, 1] = -80.0
    d["g"][:, 100, 1] = -3e4
    d["g"][:, 150:180, 1] = 0.0
    d["g"][:, 181, 1] = torch.finfo(torch.float32).min
    got, ref = _run_attn(d), _lm.attn_ref(d)
    ref["dg"] = torch.nan_to_num(ref["dg"])
    _compare(got, ref, dtype)
    # the gradient of a zero decay is zero
    assert (got["dg"][:, [0, 37, 128, 200, 255], 0].abs() <= 1e-4 * got["dg"][..., 0].abs().max()).all()
    # what stood before a reset has no influence, to the bit
    e = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    e["k"][:, :200, :], e["v"][:, :200], e["S0"] = 7.0, 3.0, e["S0"] * 5
    more = _run_attn(e, grads=False)
    assert torch.equal(more["o"][:, 200:, 0], got["o"][:, 200:, 0])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,H", [(64, 3), (128, 2)])
def test_attention_values_that_do_not_reach(D, H, dtype, bad):
    # an infinity or NaN reaches the steps after it (in the gradients' reverse walks: before it), its own head
    # and, as a value, its own column, and nothing else: not the other steps of the tile that it is in
    tol = FP32 if dtype == F32 else BF16_TWO
    d = _lm.attn_inputs(2, 300, H, H, D, dtype, True, seed=31)
    ref = _lm.attn_ref(d)
    alone = [h for h in range(H) if h != 1]

    def put(name, t):
        x = {**d, name: d[name].clone()}
        x[name][1, t, 1, 7] = bad
        return _run_attn(x)

    o = put("v", 200)["o"]
    assert not torch.isfinite(o[1, 200:, 1, 7]).any()
    check("o, other batch row", o[0], ref["o"][0], tol)
    check("o, other heads", o[:, :, alone], ref["o"][:, :, alone], tol)
    check("o, steps before", o[:, :200], ref["o"][:, :200], tol)
    others = [c for c in range(D) if c != 7]
    check("o, other columns", o[..., others], ref["o"][..., others], tol)
    dq = put("k", 200)["dq"]
    assert not torch.isfinite(dq[1, 200:, 1, 7]).any()
    check("dq, steps before", dq[:, :200], ref["dq"][:, :200], tol)
    check("dq, other heads", dq[:, :, alone], ref["dq"][:, :, alone], tol)
    dk = put("q", 70)["dk"]
    assert not torch.isfinite(dk[1, :71, 1, 7]).any()
    check("dk, steps after", dk[:, 71:], ref["dk"][:, 71:], tol)
    dv = put("grad_o", 130)["dv"]
    assert not torch.isfinite(dv[1, :131, 1, 7]).any()
    check("dv, steps after", dv[:, 131:], ref["dv"][:, 131:], tol)
    check("dv, other batch row", dv[0], ref["dv"][0], tol)


@pytest.mark.parametrize("B,T,H,Hk,D,dtype", [(1, 5000, 2, 1, 128, F32), (1, 7001, 1, 1, 64, F32), (1, 9000, 1, 1, 128, BF16),
                                              (1, 12345, 3, 3, 64, BF16), (2, 3000, 12, 12, 128, F32)])
def test_attention_many_chunks_a_segment(B, T, H, Hk, D, dtype):
    # few lanes and a long sequence: segments of several chunks, whose states are found in a pass of its own
    d = _lm.attn_inputs(B, T, H, Hk, D, dtype, True, seed=T, decay=0.05)
    _compare(_run_attn(d, grads=False), _lm.attn_ref(d, grads=False), dtype)


def test_attention_gradients_of_a_long_sequence():
    # the gradients' walks in segments and spans, against the gradients of its two halves joined at the
    # state between them
    d = _lm.cuda(_lm.attn_inputs(1, 6000, 2, 2, 128, F32, True, seed=3, decay=0.05))
    whole = api.linear_attention_bwd(d["q"], d["k"], d["v"], d["g"], d["grad_o"], d["S0"], d["grad_ST"])
    a = {n: d[n][:, :2500].contiguous() for n in ("q", "k", "v", "g", "grad_o")}
    c = {n: d[n][:, 2500:].contiguous() for n in ("q", "k", "v", "g", "grad_o")}
    _, S = api.linear_attention_fwd(a["q"], a["k"], a["v"], a["g"], d["S0"], want_state=True)
    late = api.linear_attention_bwd(c["q"], c["k"], c["v"], c["g"], c["grad_o"], S, d["grad_ST"])
    early = api.linear_attention_bwd(a["q"], a["k"], a["v"], a["g"], a["grad_o"], d["S0"], late[4])
    for n, w, x, y in zip(("dq", "dk", "dv", "dg"), whole, early, late):
        check(n, w, torch.cat([x, y], 1), 2 * FP32)
    check("dS0", whole[4], early[4], 2 * FP32)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_empty(dtype):
    S0 = torch.randn(2, 3, 64, 64, device="cuda")
    e = torch.empty(2, 0, 3, 64, device="cuda", dtype=dtype)
    g = torch.empty(2, 0, 3, device="cuda")
    o, ST = api.linear_attention_fwd(e, e, e, g, S0, want_state=True)
    assert o.shape == e.shape and torch.equal(ST, S0)
    dq, dk, dv, dg, dS0 = api.linear_attention_bwd(e, e, e, g, e, S0, S0 * 2)
    assert dg.shape == g.shape and torch.equal(dS0, S0 * 2)
    fixed = api.linear_attention_bwd(e, e, e, torch.zeros(3, device="cuda"), e)[3]
    assert torch.equal(fixed, torch.zeros(3, device="cuda"))
    z = torch.empty(0, 5, 3, 64, device="cuda", dtype=dtype)
    assert api.linear_attention_fwd(z, z, z, torch.empty(0, 5, 3, device="cuda")).shape == z.shape
    b.mgs_check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_autograd_and_scale(dtype):
    d = _lm.attn_inputs(2, 70, 4, 2, 64, dtype, True, seed=5)
    ref = _lm.attn_ref(d, scale=0.3)
    c = _lm.cuda(d)
    x = {n: c[n].requires_grad_() for n in ("q", "k", "v", "g", "S0")}
    o, ST = api.linear_attention(x["q"], x["k"], x["v"], x["g"], x["S0"], scale=0.3)
    torch.autograd.backward([o, ST], [c["grad_o"], c["grad_ST"]])
    got = {"o": o, "S_T": ST, **{"d" + n: t.grad for n, t in x.items()}}
    _compare(got, ref, dtype)
    # only the state used: its gradient alone
    o, ST = api.linear_attention(x["q"], x["k"], x["v"], x["g"], x["S0"])
    dq, dS0 = torch.autograd.grad(ST.sum(), [x["q"], x["S0"]])
    assert not dq.any() and dS0.any()


def test_attention_gradients_against_differences():
    # directional derivatives of the fp32 forward by central differences: the
    # error is eps^2 and the forward's rounding (1e-6 of the loss's terms) / eps
    d = _lm.cuda(_lm.attn_inputs(1, 140, 2, 2, 64, F32, True, seed=6))
    grads = api.linear_attention_bwd(d["q"], d["k"], d["v"], d["g"], d["grad_o"], d["S0"], d["grad_ST"])

    def loss(x):
        o, ST = api.linear_attention_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], want_state=True)
        return (o.double() * d["grad_o"].double()).sum() + (ST.double() * d["grad_ST"].double()).sum()

    eps = 2e-3
    for n, gr in zip(("q", "k", "v", "g", "S0"), grads):
        u = gr / gr.norm()  # along the gradient: its norm is the derivative
        hi, lo = loss({**d, n: d[n] + eps * u}), loss({**d, n: d[n] - eps * u})
        want = gr.double().norm().item()
        assert abs((hi - lo).item() / (2 * eps) - want) <= 5e-3 * want, n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,D,fixed", [(1, 1, 1, 64, False), (3, 4, 2, 128, False), (7, 3, 3, 64, True), (40, 6, 2, 128, True)])
def test_step_matches_the_recurrence(B, H, Hk, D, fixed, dtype):
    d = _lm.attn_inputs(B, 3, H, Hk, D, dtype, True, fixed, seed=B + D)
    ref = _lm.attn_ref(d, grads=False)
    c = _lm.cuda(d)
    N = B + 5
    slots = torch.randperm(N, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32).cuda()
    S = torch.full((N, H, D, D), 9.0, device="cuda")
    S[slots.long()] = c["S0"]
    for t in range(3):
        o = api.linear_attention_step(c["q"][:, t], c["k"][:, t], c["v"][:, t], c["g"] if fixed else c["g"][:, t], S, slots)
        check(f"o_{t}", o, ref["o"][:, t], FP32 if dtype == F32 else BF16_ONE)
    check("S", S[slots.long()], ref["S_T"], FP32)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert (S[rest] == 9.0).all()


def test_step_empty_rows():
    d = _lm.cuda(_lm.attn_inputs(4, 1, 2, 2, 64, BF16, True, seed=8))
    S = d["S0"].clone()
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")  # 4 states: the third row's is none
    o = api.linear_attention_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"][:, 0], S, slots)
    assert not o[1].any() and not o[2].any() and o[0].any() and o[3].any()
    assert torch.equal(S[1], d["S0"][1]) and torch.equal(S[3], d["S0"][3])
    with pytest.raises(ValueError, match="states"):
        api.linear_attention_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"][:, 0], S[:3])


def test_prompt_then_steps_equals_one_prompt():
    d = _lm.cuda(_lm.attn_inputs(2, 140, 2, 1, 128, BF16, False, seed=13))
    whole, ST = api.linear_attention_fwd(d["q"], d["k"], d["v"], d["g"], want_state=True)
    _, S = api.linear_attention_fwd(d["q"][:, :133], d["k"][:, :133], d["v"][:, :133], d["g"][:, :133], want_state=True)
    for t in range(133, 140):
        o = api.linear_attention_step(d["q"][:, t], d["k"][:, t], d["v"][:, t], d["g"][:, t], S)
        check("o", o, whole[:, t], BF16_TWO + BF16_ONE)
    check("S", S, ST, FP32)


def test_attention_refuses():
    d = _lm.cuda(_lm.attn_inputs(1, 8, 2, 2, 64, BF16))
    for bad, match in (({"k": d["k"].float()}, "bfloat16"), ({"g": d["g"].bfloat16()}, "float32"),
                       ({"v": d["v"][..., :32]}, "shape"), ({"g": d["g"][:, :4]}, "shape"),
                       ({"q": d["q"].transpose(2, 3).contiguous().transpose(2, 3)}, "last dimension"),
                       ({"S0": d["S0"][:, :1]}, "shape")):
        x = {**d, **bad}
        with pytest.raises(ValueError, match=match):
            api.linear_attention_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    # a head stride of 130 bytes: the library refuses, the autograd function copies
    wide = torch.zeros(1, 8, 2, 65, device="cuda", dtype=BF16)
    wide[..., :64] = d["q"]
    with pytest.raises(b.MGSError) as e:
        api.linear_attention_fwd(wide[..., :64], d["k"], d["v"], d["g"])
    assert e.value.status == b.MGS_ERR_UNSUPPORTED
    assert torch.equal(api.linear_attention(wide[..., :64], d["k"], d["v"], d["g"])[0],
                       api.linear_attention_fwd(d["q"], d["k"], d["v"], d["g"]))


# ---------------------------------------------------------------- RMS norm
def _norm_inputs(rows, N, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    return [t.to(dtype) for t in (n(rows, N), n(rows, N) * 4, n(N) * 0.3 + 1, n(rows, N), n(rows, N))]


SIZES = [(1, 8), (3, 64), (5, 77), (2, 1021), (7, 1000), (130, 256), (9, 4096), (700, 128), (2, 8200), (3, 20000), (1, 40960)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N", SIZES)
def test_norm(rows, N, dtype):
    x, res, w, gy, gr = _norm_inputs(rows, N, dtype, seed=N)
    one = FP32 if dtype == F32 else BF16_ONE
    c = [t.cuda() for t in (x, res, w, gy, gr)]
    for with_res in (True, False):
        ref = _lm.norm_ref(x, w, res if with_res else None, 1e-6, dtype, gy, gr if with_res else None)
        y, r, rstd = api.rms_norm_fwd(c[0], c[2], c[1] if with_res else None)
        dx, dw = api.rms_norm_bwd(r, c[2], rstd, c[3], c[4] if with_res else None)
        assert torch.equal(r.double().cpu(), ref["r"])
        check_rounded("y", y, ref["y"], one)
        check("rstd", rstd, ref["rstd"], FP32)
        check_rounded("dx", dx, ref["dx"], one)
        check_rounded("dw", dw, ref["dw"], one)
    b.mgs_check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N", [(20011, 13), (10007, 77), (3001, 1001), (1301, 5003), (1217, 1), (700, 8190)])
def test_norm_rows_that_start_anywhere(rows, N, dtype):
    # rows of no whole number of 16-byte pieces, more than the grid has in hand at a time; what lies behind
    # the tensors stays as it is
    x, res, w, gy, gr = (t.cuda() for t in _norm_inputs(rows, N, dtype, seed=N))
    one = FP32 if dtype == F32 else BF16_ONE
    n, pad, dt = rows * N, 64, b.MGS_F32 if dtype == F32 else b.MGS_BF16
    r, y, dx = (torch.full((n + pad,), 7.0, dtype=dtype, device="cuda") for _ in range(3))
    q8 = torch.zeros(n + pad, dtype=torch.uint8, device="cuda")
    rstd, scales = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw = torch.full((N + pad,), 7.0, dtype=dtype, device="cuda")
    b.mgs_rms_norm_fwd(x, res, w, 1e-6, r, y, rstd, rows, N, dt)
    size = b.mgs_rms_norm_bwd_workspace_size(rows, N)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    b.mgs_rms_norm_bwd(r, w, rstd, gy, gr, dx, dw, rows, N, dt, ws, size)
    r2 = torch.full_like(r, 7.0)
    b.mgs_rms_norm_fp8_fwd(x, res, w, 1e-6, r2, q8, scales, rows, N, 0, dt)
    b.mgs_check()
    ref = _lm.norm_ref(x.cpu(), w.cpu(), res.cpu(), 1e-6, dtype, gy.cpu(), gr.cpu())
    for t in (r, y, dx, r2, dw):
        assert (t[-pad:] == 7.0).all()
    assert not q8[-pad:].any()
    assert torch.equal(r[:n].view(rows, N).double().cpu(), ref["r"]) and torch.equal(r2, r)
    check_rounded("y", y[:n].view(rows, N), ref["y"], one)
    check("rstd", rstd, ref["rstd"], FP32)
    check_rounded("dx", dx[:n].view(rows, N), ref["dx"], one)
    check_rounded("dw", dw[:N], ref["dw"], one)
    check("scales", scales, ref["y"].abs().amax(-1) / 448, 1e-6)
    back = q8[:n].view(torch.float8_e4m3fn).view(rows, N).double().cpu() * scales.double().cpu()[:, None]
    # a step of e4m3 is at most 2^-3 of the value, or 2^-9 of the scale below 2^-6 of it; half of it is the error
    assert ((back - ref["y"]).abs() <= ref["y"].abs() * (2 ** -4 + 1e-5) + scales.double().cpu()[:, None] * 2 ** -10 * 1.01).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,N,group", [(1, 128, 128), (5, 77, 0), (3, 1024, 128), (3, 1024, 0), (2, 1021, 0),
                                          (11, 4096, 128), (2, 8320, 128), (1, 40960, 128), (1, 40960, 0), (600, 256, 128)])
def test_norm_fp8(rows, N, group, dtype):
    x, res, w, _, _ = _norm_inputs(rows, N, dtype, seed=N + group)
    ref = _lm.norm_ref(x, w, res, 1e-6, dtype)
    q, sc, r = api.rms_norm_fp8_fwd(x.cuda(), w.cuda(), res.cuda(), group=group)
    assert torch.equal(r.double().cpu(), ref["r"])
    y = ref["y"].view(rows, -1, group or N)
    check("scales", sc, y.abs().amax(-1) / 448, 1e-6)
    # each value is a nearest e4m3 value of y / scale, to the rounding of fp32
    val, s = q.float().double().cpu().view(y.shape), sc.double().cpu()[..., None]
    table = _lm.fp8_values()
    want = (y / s).abs()
    up = torch.bucketize(want, table).clamp(max=len(table) - 1)
    lo = table[(up - 1).clamp(min=0)]
    best = torch.minimum((want - lo).abs(), (want - table[up]).abs())
    assert ((val - y / s).abs() <= best + 1e-5 * want + 1e-9).all()
    assert (val.abs().amax(-1) == 448).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_special_rows(dtype):
    x = torch.zeros(4, 256, dtype=dtype, device="cuda")
    x[1] = 1.0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    w = torch.ones(256, dtype=dtype, device="cuda")
    y, r, rstd = api.rms_norm_fwd(x, w)
    assert not y[0].any() and (y[1].float() - 1).abs().max() < 0.01
    assert y[2, 5].isnan() and not y[2, 0].isnan() and y[3].isnan().any()
    for group in (0, 128):
        q, sc, _ = api.rms_norm_fp8_fwd(x[:2], w, group=group)
        assert not q[0].float().any() and not sc[0].any()          # a row of zeros has a scale of zero
        assert (q[1].float() == 448).all()
    assert api.rms_norm_fwd(x[:0], w)[0].shape == (0, 256)
    dx, dw = api.rms_norm_bwd(x[:0], w, rstd[:0], x[:0])
    assert dx.shape == (0, 256) and not dw.any()


def test_norm_unaligned_and_autograd():
    x, res, w, gy, gr = _norm_inputs(6, 128, BF16, seed=4)
    buf = torch.zeros(6 * 128 + 1, dtype=BF16, device="cuda")
    off = buf[1:].view(6, 128).copy_(x)                            # 2 bytes past an aligned address
    want = api.rms_norm_fwd(x.cuda(), w.cuda(), res.cuda())[0]
    assert (api.rms_norm_fwd(off, w.cuda(), res.cuda())[0].float() - want.float()).abs().max() <= 0.04
    p = [t.cuda().requires_grad_() for t in (x, res, w)]
    y, r = api.rms_norm(p[0], p[2], p[1])
    torch.autograd.backward([y, r], [gy.cuda(), gr.cuda()])
    ref = _lm.norm_ref(x, w, res, 1e-6, BF16, gy, gr)
    check_rounded("dx", p[0].grad, ref["dx"], BF16_ONE)
    check_rounded("dres", p[1].grad, ref["dx"], BF16_ONE)
    check_rounded("dw", p[2].grad, ref["dw"], BF16_ONE)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.rms_norm_fwd(x.cuda().half(), w.cuda().half())
    with pytest.raises(ValueError, match="group"):
        api.rms_norm_fp8_fwd(x.cuda()[:, :96].contiguous(), w.cuda()[:96].contiguous(), group=128)


# ---------------------------------------------------------------- clipping
def _grads(sizes, seed=0, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale).to(BF16 if i % 3 == 1 else F32).cuda() for i, n in enumerate(sizes)]


@pytest.mark.parametrize("sizes", [[1], [5, 7, 0, 3], [16384, 16385, 100003, 8], [3] * 1300, [0, 0], [2000001, 12]])
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
def test_clip(sizes, max_norm):
    grads = _grads(sizes, seed=len(sizes))
    n = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    c = min(1.0, max_norm / (n + 1e-6))
    want = [g.double() * c for g in grads]
    out = [torch.full_like(g, 3.0) for g in grads]
    keep = [g.clone() for g in grads]
    norm = api.clip_grad_norm(grads, max_norm, out=out)
    assert abs(norm.item() - n) <= 1e-5 * n
    assert all(torch.equal(g, k) for g, k in zip(grads, keep))
    norm2 = api.clip_grad_norm(grads, max_norm)
    assert norm2.item() == norm.item()
    for g, o, w in zip(grads, out, want):
        assert torch.equal(g, o)
        check_rounded("clipped", o, w, FP32 if o.dtype == F32 else BF16_ONE)
    b.mgs_check()


def test_clip_unaligned_and_special():
    buf = torch.randn(40001, device="cuda")
    g = [buf[1:20000], buf[20003:]]                                # 4 and 12 bytes past an aligned address
    want = torch.cat(g).double().norm().item()
    copy = [t.clone() for t in g]
    norm = api.clip_grad_norm(g, 1.0)
    assert abs(norm.item() - want) <= 1e-5 * want
    for t, k in zip(g, copy):
        check("clipped", t, k.double() / (want + 1e-6), FP32)
    x = torch.ones(100, device="cuda")
    x[3] = float("inf")
    assert api.clip_grad_norm([x], 1.0).isinf() and x[3].isnan() and not x[0].any()
    x = torch.ones(100, device="cuda")
    x[3] = float("nan")
    assert api.clip_grad_norm([x], 1.0).isnan() and x.isnan().all()


def test_clip_refuses():
    g = torch.randn(8, 8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        api.clip_grad_norm([g.T], 1.0)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.clip_grad_norm([g.half()], 1.0)
    with pytest.raises(ValueError, match="outputs"):
        api.clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(b.MGSError):
        api.clip_grad_norm([g], -1.0)


# ---------------------------------------------------------------- streams
def test_lm_ops_on_a_side_stream_and_repeated():
    d = _lm.cuda(_lm.attn_inputs(1, 1500, 2, 1, 128, BF16, True, seed=17))
    x, res, w, gy, _ = (t.cuda() for t in _norm_inputs(50, 512, BF16, seed=3))
    grads = _grads([70000, 300, 9])

    def run(stream=None):
        o, ST = api.linear_attention_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], want_state=True, stream=stream)
        r = api.linear_attention_bwd(d["q"], d["k"], d["v"], d["g"], d["grad_o"], d["S0"], d["grad_ST"], stream=stream)
        y, rr, rstd = api.rms_norm_fwd(x, w, res, stream=stream)
        n = api.rms_norm_bwd(rr, w, rstd, gy, stream=stream)
        out = [torch.empty_like(t) for t in grads]
        norm = api.clip_grad_norm(grads, 0.5, out=out, stream=stream)
        return [o, ST, *r, y, *n, norm, *out]

    ref = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.empty(64 << 20, device="cuda")
    with torch.cuda.stream(side):
        busy.normal_()
        inside = run(side.cuda_stream)
    outside = run(side)           # the stream named, another one current
    side.synchronize()
    b.mgs_check()
    for p, q, s in zip(ref, inside, outside):
        assert torch.equal(p, q) and torch.equal(p, s)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lm_ops_captured_in_a_graph(dtype):
    # launches that are set up early keep their order in a graph; replayed on other inputs it gives their outputs
    d = _lm.cuda(_lm.attn_inputs(1, 2300, 3, 1, 64, dtype, True, seed=41, decay=0.05))
    x, res, w, gy, _ = (t.cuda() for t in _norm_inputs(300, 512, dtype, seed=5))
    grads = _grads([70000, 300, 9])
    names = ("q", "k", "v", "g", "grad_o", "S0", "grad_ST")

    def run():
        o, ST = api.linear_attention_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], want_state=True)
        r = api.linear_attention_bwd(d["q"], d["k"], d["v"], d["g"], d["grad_o"], d["S0"], d["grad_ST"])
        y, rr, rstd = api.rms_norm_fwd(x, w, res)
        n = api.rms_norm_bwd(rr, w, rstd, gy)
        out = [torch.empty_like(t) for t in grads]
        return [o, ST, *r, y, *n, api.clip_grad_norm(grads, 0.5, out=out), *out]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    other = _lm.cuda(_lm.attn_inputs(1, 2300, 3, 1, 64, dtype, True, seed=42, decay=0.05))
    for n in names:
        d[n].copy_(other[n])
    x.mul_(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, e in zip(got, run()):
        assert torch.equal(a, e)
    b.mgs_check()
