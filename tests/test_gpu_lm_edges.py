"""GPU tests of the language-model operators at the edges of what they take:
broadcast inputs on a named stream, and the like; references as in
test_gpu_lm_ops."""
import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api
from scan_linear_recurrences_gb300.build import build

from . import _lm

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


# ---------------------------------------------------------------- linear attention
@pytest.mark.parametrize("address", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_broadcast_inputs_on_a_named_stream(dtype, address):
    # q the same for all steps, grad_o for all steps and sequences: where the call copies them, the copies are
    # the named stream's too, whatever the current one is busy with
    d = _lm.cuda(_lm.attn_inputs(2, 300, 4, 2, 64, dtype, False, seed=51))
    q = d["q"][:, :1].expand(2, 300, 2, 64)
    go = d["grad_o"][:1, :1].expand(2, 300, 4, 64)
    want = [api.linear_attention_fwd(q, d["k"], d["v"], d["g"]), *api.linear_attention_bwd(q, d["k"], d["v"], d["g"], go)]
    side = torch.cuda.Stream()
    named = side.cuda_stream if address else side
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)  # some milliseconds on the current stream
    got = [api.linear_attention_fwd(q, d["k"], d["v"], d["g"], stream=named),
           *api.linear_attention_bwd(q, d["k"], d["v"], d["g"], go, stream=named)]
    torch.full((1 << 20,), 9.0, dtype=dtype, device="cuda")  # takes what memory the current stream has been given back
    b.mgs_check(named)
    torch.cuda.synchronize()
    for x, y in zip(got[:-1], want[:-1]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("name", ["q", "k"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_broadcast_queries_and_keys_run_as_dense_ones(dtype, name):
    # the tensor functions copy them where no tensor map describes them: the same kernels, the same bits
    d = _lm.cuda(_lm.attn_inputs(2, 200, 2, 2, 64, dtype, True, seed=52))
    d[name] = d[name][:, :1].expand(2, 200, 2, 64)
    args = lambda x: (x["q"], x["k"], x["v"], x["g"])  # noqa: E731
    e = {**d, name: d[name].contiguous()}
    assert torch.equal(api.linear_attention_fwd(*args(d), d["S0"]), api.linear_attention_fwd(*args(e), d["S0"]))
    for x, y in zip(api.linear_attention_bwd(*args(d), d["grad_o"], d["S0"], d["grad_ST"]),
                    api.linear_attention_bwd(*args(e), d["grad_o"], d["S0"], d["grad_ST"])):
        assert torch.equal(x, y)


def _through_the_c_entry(d, scale):
    """Forward and backward with the tensors' own strides, zero ones among them."""
    c = _lm.cuda({n: t for n, t in d.items() if isinstance(t, torch.Tensor)})
    for n in ("q", "k", "v", "grad_o"):  # .cuda() keeps no zero strides
        lead = tuple(slice(0, 1) if st == 0 else slice(None) for st in d[n].stride())
        c[n] = d[n][lead].contiguous().cuda().expand(d[n].shape)
    (B, T, Hk, D), H, dtype = d["q"].shape, d["v"].shape[2], d["q"].dtype
    fixed = d["g"].dim() == 1
    shape = b.mgs_attention_shape(B, T, H, Hk, D, b.MGS_F32 if dtype == F32 else b.MGS_BF16, fixed, scale,
                                  *(c[n].stride()[:3] for n in ("q", "k", "v")),
                                  (0, 0, 1) if fixed else c["g"].stride(), c["grad_o"].stride()[:3])
    new = lambda *s, dt=dtype: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    out = {"o": new(B, T, H, D), "S_T": new(B, H, D, D, dt=F32), "dq": new(B, T, Hk, D), "dk": new(B, T, Hk, D),
           "dv": new(B, T, H, D), "dg": new(*d["g"].shape, dt=F32), "dS0": new(B, H, D, D, dt=F32)}
    ws = []
    for backward in (False, True):
        n = b.mgs_linear_attention_workspace_size(shape, backward)
        ws.append((torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"), n))
    S0, gST = c.get("S0"), c.get("grad_ST")
    b.mgs_linear_attention_fwd(shape, c["q"], c["k"], c["v"], c["g"], S0, out["o"], out["S_T"], *ws[0])
    b.mgs_linear_attention_bwd(shape, c["q"], c["k"], c["v"], c["g"], S0, c["grad_o"], gST, out["dq"], out["dk"],
                               out["dv"], out["dg"], out["dS0"] if S0 is not None else None, *ws[1])
    b.mgs_check()
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,H,Hk,S0,fixed,name,dim", [
    (2, 1, 2, 2, True, False, "q", 0), (2, 17, 2, 1, True, False, "k", 1), (1, 60, 4, 2, False, True, "q", 2),
    (2, 300, 2, 2, True, False, "k", 0), (3, 333, 3, 3, True, True, "q", 1),  # fp32: two spans of the decay's gradient
    (1, 1300, 1, 1, True, False, "k", 1), (1, 1500, 2, 1, False, False, "q", 1),  # segments; bf16: two spans
    (2, 200, 2, 2, True, False, "v", 1), (2, 150, 4, 2, True, False, "grad_o", 0),  # (bf16 alone takes the recurrence)
])
def test_recurrence_kernel_through_the_c_entry(B, T, H, Hk, S0, fixed, name, dim, D, dtype):
    # a stride of zero, which no tensor map has: the walk that is the recurrence itself, in both directions, with
    # its row products, kept states and segments
    d = _lm.attn_inputs(B, T, H, Hk, D, dtype, S0, fixed, seed=B + T + D, decay=0.05)
    d[name] = d[name].narrow(dim, 0, 1).expand(d[name].shape)
    got, ref = _through_the_c_entry(d, D ** -0.5), _lm.attn_ref(d)
    tol = _lm.FP32 if dtype == F32 else _lm.BF16_TWO
    for n, r in ref.items():
        _lm.check(n, got[n], r, _lm.FP32 if n in ("S_T", "dg", "dS0") else tol)


@pytest.mark.parametrize("B,T,H,Hk,D", [(2, 300, 3, 3, 64), (1, 700, 4, 2, 64), (2, 300, 2, 2, 128), (1, 700, 4, 1, 128),
                                        (1, 5000, 2, 2, 128), (3, 1, 2, 2, 64), (40, 129, 4, 4, 64), (40, 129, 4, 4, 128)])
@pytest.mark.parametrize("resets", [False, True])
def test_bf16_outputs_are_rounded_once(B, T, H, Hk, D, resets):
    # what is computed of bf16 inputs is held to 2^-17 and better before the output's own rounding, sums of many
    # strong decays included.  Granted that to 2^-14 of the output, an element differs from the rounded reference
    # by a step (2^-8) where the reference is as near as that to a tie, one of 64: 2^-11 of the whole
    d = _lm.attn_inputs(B, T, H, Hk, D, BF16, True, seed=D + T, decay=0.3)
    if resets:
        d["g"][:, ::3] = -100.0  # from the sums of g only the differences between near steps count
    c, grads = _lm.cuda(d), T <= 700 and B < 40
    ref = _lm.attn_ref(d, grads=grads)
    got = {"o": api.linear_attention_fwd(c["q"], c["k"], c["v"], c["g"], c["S0"])}
    if grads:
        r = api.linear_attention_bwd(c["q"], c["k"], c["v"], c["g"], c["grad_o"], c["S0"], c["grad_ST"])
        got.update(zip(("dq", "dk", "dv"), r))
    b.mgs_check()
    for n, x in got.items():
        _lm.check(n, x, ref[n], _lm.BF16_ONE)
        _lm.check_rounded(n, x, ref[n], 2.0 ** -11)


def test_prompt_and_tokens_agree_to_one_rounding():
    d = _lm.cuda(_lm.attn_inputs(3, 150, 4, 2, 128, BF16, False, seed=54))
    whole = api.linear_attention_fwd(d["q"], d["k"], d["v"], d["g"])
    _, S = api.linear_attention_fwd(*(d[n][:, :130] for n in ("q", "k", "v", "g")), want_state=True)
    for t in range(130, 150):
        o = api.linear_attention_step(*(d[n][:, t] for n in ("q", "k", "v", "g")), S)
        _lm.check("o", o, whole[:, t], 2.0 ** -11)  # the same value rounded, but where it is near a tie


def _dg64(d, scale):
    """The decay's gradient in 64 bits: dg_t = <R_t, e^{g_t} S_{t-1}> from dg_t - dg_{t+1} = <q_t, dq_t> - <k_t, dk_t>."""
    q, k, v, go = (d[n].double().cuda() for n in ("q", "k", "v", "grad_o"))
    (B, T, H, D), a = q.shape, d["g"].double().cuda().exp()[:, None, None]
    S, x = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda"), torch.empty(B, T, H, dtype=torch.float64, device="cuda")
    R = torch.zeros_like(S)
    for t in range(T):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        x[:, t] = scale * ((S @ go[:, t, :, :, None])[..., 0] * q[:, t]).sum(-1)
    for t in range(T - 1, -1, -1):
        R = R + scale * q[:, t, :, :, None] * go[:, t, :, None, :]
        x[:, t] -= ((R @ v[:, t, :, :, None])[..., 0] * k[:, t]).sum(-1)
        R = a * R
    return x.flip(1).cumsum(1).flip(1)


@pytest.mark.parametrize("seed", range(10))
@pytest.mark.parametrize("D", [64, 128])
def test_gradient_of_a_fixed_decay(D, seed):
    # one number for thousands of steps, whose gradients cancel in it: the more, the faster the decay
    d = _lm.attn_inputs(8, 1000, 8, 8, D, BF16, False, True, seed=seed, decay=0.5)
    c = _lm.cuda(d)
    got = api.linear_attention_bwd(c["q"], c["k"], c["v"], c["g"], c["grad_o"])[3]
    b.mgs_check()
    _lm.check("dg", got, _dg64(d, D ** -0.5).sum((0, 1)), _lm.FP32)


def test_step_on_a_state_that_autograd_has_saved():
    # the state of a prompt is saved for the gradients; a token that is stepped on it in place would falsify them
    d = _lm.cuda(_lm.attn_inputs(1, 20, 2, 2, 64, BF16, True, seed=53))
    q = d["q"].requires_grad_()
    o, _ = api.linear_attention(q, d["k"], d["v"], d["g"], d["S0"])
    api.linear_attention_step(d["q"][:, 0].detach(), d["k"][:, 0], d["v"][:, 0], d["g"][:, 0], d["S0"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        o.sum().backward()


def _filled(monkeypatch):
    """From here on torch.empty's memory holds sevens: what a call leaves alone shows."""
    empty = torch.empty

    def full(*a, **k):
        t = empty(*a, **k)
        return t.fill_(7) if t.is_cuda else t
    monkeypatch.setattr(torch, "empty", full)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_without_value_heads(monkeypatch, dtype):
    q = torch.randn(2, 5, 2, 64, device="cuda", dtype=dtype)
    v, g = q[:, :, :0], torch.zeros(2, 5, 0, device="cuda")
    _filled(monkeypatch)
    dq, dk, dv, dg, _ = api.linear_attention_bwd(q, q, v, g, v)
    b.mgs_check()
    assert dq.shape == q.shape and not dq.any() and not dk.any() and dv.numel() == dg.numel() == 0


def test_norm_of_rows_of_nothing(monkeypatch):
    x, w = torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda")
    _filled(monkeypatch)
    y, r, rstd = api.rms_norm_fwd(x, w)
    q, sc, _ = api.rms_norm_fp8_fwd(x, w)
    dx, dw = api.rms_norm_bwd(r, w, rstd, y)
    b.mgs_check()
    assert y.shape == q.shape == dx.shape == (3, 0) and dw.shape == (0,)
    assert rstd.isnan().all() and not sc.any()  # the mean of nothing, the largest of nothing


# ---------------------------------------------------------------- RMS norm in 8 bits
def _fp8(x, w, group, aligned=True):
    """q as numbers, the scales with a column for each q, both in 64 bits; x 16 bytes aligned, or not."""
    buf = torch.zeros(x.numel() + 8, dtype=x.dtype, device="cuda")
    xc = buf[8 if aligned else 1:][:x.numel()].view(x.shape).copy_(x)
    q, sc, _ = api.rms_norm_fp8_fwd(xc, w.cuda(), group=group)
    b.mgs_check()
    return q.float().double().cpu(), sc.double().cpu().repeat_interleave(group or x.shape[1], 1)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tiny", [1e-37, 1e-40, 1e-44])
def test_norm_fp8_of_the_smallest_numbers(tiny, dtype, group, aligned):
    # a group's (or the whole row's) values so small that the scale is subnormal, or zero; zeros among them
    gen = torch.Generator().manual_seed(61)
    x = torch.randn(5, 384, generator=gen).to(dtype)
    x[:, ::7] = 0
    w = torch.randn(384, generator=gen) + 3
    w[128 if group else 0:256 if group else 384] *= tiny
    w = w.to(dtype)
    q, s = _fp8(x, w, group, aligned)
    y = _lm.norm_ref(x, w, None, 1e-6, dtype)["y"]
    want = y.view(5, -1, group or 384).abs().amax(-1).repeat_interleave(group or 384, 1) / 448
    unit = 2.0 ** -149  # fp32's smallest step; y, the maximum and the scale are each a rounding to it
    assert ((s - want).abs() <= want * 1e-5 + 2 * unit).all()
    # half a step of e4m3 (2^-3 of the value, or 2^-9 below 2^-6), and the scale's own error times q
    err = y.abs() * (2 ** -4 + 1e-5) + s * 2 ** -10 * 1.01 + 448 * 2 * unit
    assert ((q * s - y).abs() <= err).all()
    assert not q[:, ::7].any() and not q[s == 0].any() and (s == 0).any() == (tiny == 1e-44)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_fp8_of_infinities_and_nan(dtype, group, aligned):
    # as the formula in fp32 has them: a NaN makes its scale NaN (all of a row's: the row's own norm is NaN
    # or infinite), an infinite weight an infinite scale and zeros beside it
    gen = torch.Generator().manual_seed(62)
    x = torch.randn(5, 384, generator=gen).to(dtype)
    x[1, 5], x[2, 200], x[3, 7] = float("nan"), float("inf"), -float("inf")
    for column, value in ((None, 1.0), (300, float("nan")), (140, float("inf"))):
        w = torch.randn(384, generator=gen).to(dtype)
        if column is not None:
            w[column] = value
        q, s = _fp8(x, w, group, aligned)
        r = x.float()
        y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        sc = (y.view(5, -1, group or 384).abs().amax(-1) / 448).repeat_interleave(group or 384, 1)
        z = (y / torch.where(sc > 0, sc, torch.ones_like(sc))).clamp(-448, 448)
        assert torch.equal(s.isnan(), sc.isnan()) and torch.equal(q.isnan(), z.isnan())
        assert torch.equal(s.isinf(), sc.isinf())
        fine = sc.isfinite()
        assert ((s - sc).abs()[fine] <= 1e-5 * sc[fine]).all()
        number = ~z.isnan()  # half a step of e4m3, and the rounding of fp32
        assert ((q - z)[number].abs() <= z[number].abs() * (2 ** -4 + 1e-5) + 2 ** -10 * 1.01).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N", [13, 56, 64, 77, 128])
@pytest.mark.parametrize("rows", [1, 6, 9, 16, 23, 12345])
def test_norm_rows_that_do_not_fill_a_block(rows, N, dtype):
    # several rows a warp, the last block's rows not all there
    gen = torch.Generator().manual_seed(rows + N)
    x, res, gy, gr = (torch.randn(rows, N, generator=gen).to(dtype) for _ in range(4))
    w = torch.randn(N, generator=gen).to(dtype)
    y, r, rstd = api.rms_norm_fwd(x.cuda(), w.cuda(), res.cuda())
    dx, dw = api.rms_norm_bwd(r, w.cuda(), rstd, gy.cuda(), gr.cuda())
    q, sc, _ = api.rms_norm_fp8_fwd(x.cuda(), w.cuda(), res.cuda())
    b.mgs_check()
    ref = _lm.norm_ref(x, w, res, 1e-6, dtype, gy, gr)
    one = _lm.FP32 if dtype == F32 else _lm.BF16_ONE
    for name, got in (("y", y), ("dx", dx), ("dw", dw)):
        _lm.check_rounded(name, got, ref[name], one)
    _lm.check("rstd", rstd, ref["rstd"], _lm.FP32)
    _lm.check("scales", sc[:, 0], ref["y"].abs().amax(-1) / 448, _lm.FP32)
    _lm.check("q", q.float() * sc, ref["y"], 2 ** -4)  # each value within half a step of e4m3
