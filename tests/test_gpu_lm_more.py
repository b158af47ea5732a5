"""GPU tests of the gated recurrence, the norm of queries and keys with its
rotation, and the embedding, against 64-bit formulas.

Tolerances.  Elementwise: one rounding to the output's type, and beside it an
error of the fp32 computation, in units u = 2^-24.
Gated recurrence: a gate's z and a come out of an exponential of relative error
|gate| u + 4 u, a sum and a reciprocal (3 u): at gates up to 10 less than 20 u
each.  A state sums contributions that have passed at most as many steps as the
channel remembers, each step adding an error of 20 u z (of a = 1 / (1 + e), e
erring by e / (1 + e) = z of it) and 3 u of its own roundings; with memories of up
to 100 steps (gates down to -5) no more than 400 u of the largest state or
gradient in that channel, which is what its contributions are bounded by.
Norm: the sum of up to 256 squares 16 u at most, rsqrt and products 6 u, the rotation's two
products and sum 3 u, the table's rounding 1 u: 32 u of the pair's length, which is
at most the head's.  The gradient takes two such factors and a mean: 100 u of the
largest.  Sums over tokens: (count + 100) u of the sum of magnitudes at worst, less than
1e-5 of a weight gradient's norm.
Embedding: rows in order, one product a row; sums (count + 2) u of the terms' magnitudes.
"""
import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api
from scan_linear_recurrences_gb300.build import build

from . import _lm_more as m
from ._lm import cuda

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    build()
    b.lib()
    yield
    b.mgs_check()


# ---------------------------------------------------------------- gated recurrence
def _views(d):
    """On the GPU with the strides that they have here (.cuda() makes tensors dense)."""
    out = cuda({n: t for n, t in d.items() if not isinstance(t, torch.Tensor)})
    for n, t in d.items():
        if not isinstance(t, torch.Tensor):
            continue
        size = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride())) if t.numel() else 0
        if not size:
            out[n] = torch.empty(t.shape, dtype=t.dtype, device="cuda")
            continue
        base = torch.as_strided(t, (t.storage_offset() + size,), (1,), 0).cuda()
        out[n] = base.as_strided(t.shape, t.stride(), t.storage_offset())
    return out


def _gated_run(c, bwd=True, stream=None):
    h, hT, carries = api.gated_scan_fwd(c["gate"], c["value"], c["h0"], c["positive"], want_carries=True, stream=stream)
    out = {"h": h, "h_T": hT, "carries": carries}  # (kept until the stream is done with them)
    if bwd:
        out["dgate"], out["dvalue"], dh0 = api.gated_scan_bwd(c["gate"], c["value"], carries, c["grad_h"], c["grad_hT"],
                                                              c["positive"], need_dh0=True, stream=stream)
        out["dh0"] = dh0
    return out


def _gated_check(got, ref, err=400 * U):
    for n, r in ref.items():
        if n == "lam":
            continue
        top = r.abs().amax(1, keepdim=True) if r.dim() == 3 and r.shape[1] else r.abs()
        if n in ("h_T", "dh0") and r.numel():  # of the largest on the way
            top = ref["h" if n == "h_T" else "lam"].abs().amax(1) if ref["h"].shape[1] else top
            top = torch.maximum(top, r.abs())
        m.check_each(n, got[n], r, err * top)


SIZES = [(1, 1, 1), (2, 1, 8), (1, 2, 3), (3, 7, 5), (2, 63, 16), (2, 64, 16), (2, 65, 16), (1, 100, 130), (4, 129, 64),
         (1, 300, 257), (2, 700, 66), (1, 2500, 34), (5, 513, 128), (1, 128, 1000), (33, 40, 96), (1, 4500, 64),
         (300, 70, 64), (2, 1025, 1026)]


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D", SIZES)
def test_gated(B, T, D, dtype, positive):
    d = m.gated_inputs(B, T, D, dtype, h0=(T + D) % 3 != 0, positive=positive, seed=B + T + D)
    _gated_check(_gated_run(_views(d)), m.gated_ref(d))


@pytest.mark.parametrize("D", [64, 63, 66])
@pytest.mark.parametrize("T", [1, 64, 65, 127, 129, 192, 335])
@pytest.mark.parametrize("B", [120, 250])
def test_gated_many_lanes(B, T, D):
    # no clusters, and in bf16 a forward whose tiles hold two of the kept states
    d = m.gated_inputs(B // -(-D // 64), T, D, BF16, h0=T % 2 == 0, seed=B + T + D)
    _gated_check(_gated_run(_views(d)), m.gated_ref(d))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_long_memory(dtype):
    # one channel each of a memory of a step, some hundred and some thousand steps, over a long sequence: with gates
    # down to -8 the error's bound of contributions is 3000 steps of 3 u, and a's 20 u z of each
    gen = torch.Generator().manual_seed(1)
    B, T, D = 1, 9000, 6
    d = m.gated_inputs(B, T, D, dtype, seed=2, shift=0.0)
    d["gate"] = (d["gate"].float() * 0.3 + torch.tensor([3.0, 0, -2, -4, -6, -8])).to(dtype)
    d["grad_h"] = torch.randn(B, T, D, generator=gen).to(dtype)
    _gated_check(_gated_run(_views(d)), m.gated_ref(d), 10000 * U)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("how", ["odd start", "odd stride", "broadcast steps", "broadcast batch", "one vector", "swapped"])
def test_gated_strides(how, dtype):
    B, T, D = 3, 150, 64
    d = m.gated_inputs(B, T, D, dtype, seed=7)
    gen = torch.Generator().manual_seed(8)
    if how == "odd start":
        big = torch.randn(B, T, 2 * D + 3, generator=gen).to(dtype)
        d["gate"], d["value"] = big[..., 1:D + 1], big[..., D + 2:2 * D + 2]
    elif how == "odd stride":
        big = torch.randn(B, T, 2 * D + 1, generator=gen).to(dtype)
        d["gate"], d["value"], d["grad_h"] = big[..., :D], big[..., D:2 * D], big[..., 1:D + 1]
    elif how == "broadcast steps":
        d["gate"], d["grad_h"] = d["gate"][:, :1].expand(B, T, D), d["grad_h"][:, 3:4].expand(B, T, D)
    elif how == "broadcast batch":
        d["value"] = d["value"][:1].expand(B, T, D)
    elif how == "one vector":
        d["gate"] = d["gate"][0, 0].expand(B, T, D)
    else:  # [T,B,D] in memory
        d["value"] = d["value"].transpose(0, 1).contiguous().transpose(0, 1)
    c = _views(d)
    assert c["gate"].stride() == d["gate"].stride() and c["grad_h"].stride() == d["grad_h"].stride()
    _gated_check(_gated_run(c), m.gated_ref(d))


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D", [(200, 32), (70, 33), (3000, 64)])
def test_gated_masked_steps(T, D, dtype, positive):
    # gates of -inf: the step is not there, whatever its value (NaN, infinities); some rows are masked throughout
    d = m.gated_inputs(3, T, D, dtype, positive=positive, seed=9, halves=False)
    gen = torch.Generator().manual_seed(10)
    off = torch.rand(3, T, D, generator=gen) < 0.3
    off[1] = True
    d["gate"][off] = -torch.inf
    for i, x in enumerate((torch.nan, torch.inf, -torch.inf, 3e38)):
        d["value"][off & (torch.arange(T) % 5 == i)[:, None]] = x
    # where all steps are masked nothing is forgotten: dh0 is the sum of T gradients (a = 1), each addition rounding by
    # u of the partial sum, which is an L_t: T u of the largest L beside the bound of channels that forget
    got, ref = _gated_run(_views(d)), m.gated_ref(d)
    _gated_check(got, ref, (400 + T) * U)
    for n in ("dgate", "dvalue"):
        assert not got[n].cpu()[off].any()
    assert torch.equal(got["h_T"][1].cpu(), d["h0"][1])
    # without a state: zeros
    d["h0"] = None
    assert not _gated_run(_views(d))["h"][1].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_new_starts(dtype):
    # a gate of +inf: the state is the candidate, and nothing flows back past it
    d = m.gated_inputs(2, 400, 64, dtype, seed=11, halves=False)
    for t in (0, 1, 63, 64, 130, 399):
        d["gate"][:, t] = torch.inf
    got, ref = _gated_run(_views(d)), m.gated_ref(d)
    _gated_check(got, ref)
    assert not got["dh0"].any()
    parts = [_gated_run(_views({**d, "gate": d["gate"][:, a:z], "value": d["value"][:, a:z], "grad_h": d["grad_h"][:, a:z]}),
                        bwd=False)["h"] for a, z in ((64, 130), (130, 399))]
    want = ref["h"][:, 64:399]
    m.check_each("parts", torch.cat(parts, 1), want, 400 * U * want.abs().amax())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D", [(300, 32), (2300, 34), (90, 7)])
@pytest.mark.parametrize("what", ["value inf", "value nan", "gate nan", "grad nan", "h0 inf"])
def test_gated_non_finite(what, T, D, dtype):
    # reaches its own channel from its step on (a gradient: up to its step), nothing else
    d = m.gated_inputs(2, T, D, dtype, seed=12, halves=False)
    t, ch = T * 2 // 3, D // 2
    if what == "value inf":
        d["value"][0, t, ch] = torch.inf
    elif what == "value nan":
        d["value"][0, t, ch] = torch.nan
    elif what == "gate nan":
        d["gate"][0, t, ch] = torch.nan
    elif what == "grad nan":
        d["grad_h"][0, t, ch] = torch.nan
    else:
        d["h0"][0, ch] = torch.inf
    got = {n: x.cpu() for n, x in _gated_run(_views(d)).items()}
    ref = m.gated_ref(d)
    for n in ("h", "dgate", "dvalue"):
        bad = ~torch.isfinite(ref[n])
        # what the formula leaves finite is finite and right
        g, r = got[n].double().masked_fill(bad, 0), ref[n].masked_fill(bad, 0)
        m.check_each(n, g.to(dtype), r, 400 * U * r.abs().amax(1, keepdim=True))
    first = 0 if what == "h0 inf" else T if what == "grad nan" else t
    assert torch.isfinite(got["h"][0, :first, ch]).all()
    if what in ("value nan", "gate nan"):
        assert torch.isnan(got["h"][0, t:, ch]).all() and torch.isnan(got["h_T"][0, ch])
    if what == "grad nan":
        assert torch.isnan(got["dvalue"][0, :t + 1, ch]).all() and torch.isnan(got["dh0"][0, ch])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_far_gates(dtype):
    # z and a to their own last digits where they are tiny: gates up to 80 in magnitude
    k = torch.linspace(-80, 80, 321)
    d = {"gate": k.expand(1, 1, -1).to(dtype), "value": torch.full((1, 1, 321), -0.75).to(dtype), "h0": torch.full((1, 321), 2.0),
         "grad_h": torch.ones(1, 1, 321).to(dtype), "grad_hT": None, "positive": True}
    d["gate"] = d["gate"].contiguous()
    got, ref = _gated_run(_views(d)), m.gated_ref(d)
    for n in ("dgate", "dvalue", "dh0"):  # |gate| u of the exponential and 20 u
        m.check_each(n, got[n], ref[n], (d["gate"].double().abs().reshape(ref[n].shape) + 20) * U * ref[n].abs())


def test_gated_smallest_negative_values():
    # the candidate's slope is that of its own side of zero, however near
    v = torch.tensor([0.0, -0.0, -1e-38, 1e-38, -1e-20, -3e-9, 3e-9, -1e-6]).expand(1, 1, 8).contiguous()
    for dtype in (F32, BF16):
        d = {"gate": torch.zeros(1, 1, 8, dtype=dtype), "value": v.to(dtype), "h0": None, "grad_h": torch.ones(1, 1, 8, dtype=dtype),
             "grad_hT": None, "positive": True}
        _gated_check(_gated_run(_views(d)), m.gated_ref(d), 20 * U)


@pytest.mark.parametrize("B,T,D", [(0, 5, 8), (2, 0, 8), (2, 5, 0), (0, 0, 0)])
def test_gated_empty(B, T, D):
    d = m.gated_inputs(B, T, D)
    got = _gated_run(_views(d))
    assert got["h"].shape == (B, T, D) and torch.equal(got["h_T"].cpu(), d["h0"]) and torch.equal(got["dh0"].cpu(), d["grad_hT"])
    assert not _gated_run(_views({**d, "h0": None, "grad_hT": None}))["h_T"].any()


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,N,D", [(1, 1, 1), (3, 5, 64), (7, 7, 33), (200, 230, 130), (2, 3, 2048)])
def test_gated_step(B, N, D, dtype, positive):
    d = m.gated_inputs(B, 1, D, dtype, positive=positive, seed=B + D)
    gen = torch.Generator().manual_seed(3)
    state = torch.randn(N, D, generator=gen)
    slots = torch.randperm(N, generator=gen)[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, N  # empty rows
    live = (slots >= 0) & (slots < N)
    ref = m.gated_ref({**d, "h0": state[slots.clamp(0, N - 1).long()]}, grads=False)["h"][:, 0] * live[:, None]
    c, s = _views(d), state.cuda()
    h = api.gated_scan_step(c["gate"][:, 0], c["value"][:, 0], s, slots.cuda(), positive)
    m.check_each("h", h, ref, 30 * U * (ref.abs() + 1))
    want = state.double()
    want[slots[live].long()] = ref[live]
    m.check_each("state", s, want, 30 * U * (want.abs() + 1))
    untouched = torch.ones(N, dtype=torch.bool)
    untouched[slots[live].long()] = False
    assert torch.equal(s.cpu()[untouched], state[untouched])
    # without slots, into a given output
    if N == B:
        s, out = state.cuda(), torch.full((B, D), 7.0, dtype=dtype, device="cuda")
        assert api.gated_scan_step(c["gate"][:, 0], c["value"][:, 0], s, positive=positive, out=out) is out
        ref = m.gated_ref({**d, "h0": state}, grads=False)["h"][:, 0]
        m.check_each("out", out, ref, 30 * U * (ref.abs() + 1))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_prompt_and_steps_agree(dtype):
    d = _views(m.gated_inputs(4, 150, 96, dtype, h0=False, seed=21))
    whole, hT = api.gated_scan_fwd(d["gate"], d["value"])
    _, state = api.gated_scan_fwd(d["gate"][:, :140], d["value"][:, :140])
    for t in range(140, 150):
        h = api.gated_scan_step(d["gate"][:, t], d["value"][:, t], state)
        m.check_each("h", h, whole[:, t].float(), (400 * U + m.HALF[dtype]) * whole[:, t].abs().amax().item())
    m.check_each("state", state, hT, 400 * U * hT.abs().amax().item())
    # pieces, each from the state before
    h1, s1 = api.gated_scan_fwd(d["gate"][:, :77], d["value"][:, :77])
    h2, s2 = api.gated_scan_fwd(d["gate"][:, 77:], d["value"][:, 77:], s1)
    m.check_each("pieces", s2, hT, 400 * U * hT.abs().amax().item())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_gradients_through_autograd_and_against_differences(dtype):
    d = m.gated_inputs(2, 200, 40, dtype, seed=22)
    c = _views(d)
    both = torch.cat([c["gate"], c["value"]], -1).requires_grad_()
    h0 = c["h0"].requires_grad_()
    h, hT = api.gated_scan(*both.split(40, -1), h0)
    loss = (h.float() * c["grad_h"].float()).sum() + (hT * c["grad_hT"]).sum()
    loss.backward()
    ref = m.gated_ref(d)
    _gated_check({"dgate": both.grad[..., :40], "dvalue": both.grad[..., 40:], "h": h, "h_T": hT, "dh0": h0.grad}, ref)
    if dtype == F32:
        # against differences of the library's own forward, in a step of 2^-7: truncation 2^-14 of the third derivative,
        # rounding 1e-6 / 2^-7.  With values as they are: the positive candidate's slope jumps at zero, where no
        # difference is a derivative (it is held to the formula's above).
        gen = torch.Generator(device="cuda").manual_seed(5)
        u, eps = torch.randn(both.shape, generator=gen, device="cuda"), 2.0 ** -7

        def at(x):
            h, hT = api.gated_scan(*x.split(40, -1), h0.detach(), positive=False)
            return (h.double() * c["grad_h"]).sum() + (hT.double() * c["grad_hT"]).sum()

        both.grad = None
        at(both).backward()
        x = both.detach()
        got = (at(x + eps * u) - at(x - eps * u)) / (2 * eps)
        want = (both.grad.double() * u).sum()
        size = (both.grad.double() * u).norm()
        assert abs(got - want) <= 1e-2 * size


def test_gated_gradient_of_a_broadcast_value():
    d = _views(m.gated_inputs(3, 70, 16, seed=23))
    v = d["value"][0, 0].clone().requires_grad_()
    h, _ = api.gated_scan(d["gate"], v.expand(3, 70, 16))
    h.sum().backward()
    c = {**{n: x.cpu() if isinstance(x, torch.Tensor) else x for n, x in d.items()}, "h0": None, "grad_hT": None}
    c["value"], c["grad_h"] = v.detach().cpu().expand(3, 70, 16), torch.ones(3, 70, 16)
    ref = m.gated_ref(c)["dvalue"].sum((0, 1))
    m.check_each("dv", v.grad, ref, 1000 * U * ref.abs().amax())


# ---------------------------------------------------------------- norm of queries and keys
def _qk_table(d):
    return api.rotary_table(d["rows"], d["R"]) if d["R"] else None


def _qk_run(c, table, eps=1e-6, bwd=True, stream=None):
    opts = {"table": table, "positions": c["at"], "eps": eps, "interleaved": c["interleaved"], "stream": stream}
    q, k = api.qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], **opts)
    out = {"q": q, "k": k}
    if bwd:
        dq, dk, dwq, dwk = api.qk_norm_bwd(c["q"], c["k"], c["wq"], c["wk"], c["grad_q"], c["grad_k"], **opts)
        out.update(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    return out


def _qk_check(got, ref, d):
    for n in ("q", "k"):
        r = ref[n]
        top = r.abs().amax(-1, keepdim=True) if r.numel() else 0
        m.check_each(n, got[n], r, 32 * U * 4 * top)  # a pair's length is up to sqrt 2, a head's norm 4 times its largest
        if "d" + n in ref:
            r = ref["d" + n]
            m.check_each("d" + n, got["d" + n], r, 100 * U * 16 * (r.abs().amax(-1, keepdim=True) if r.numel() else 0))
            if d["w" + n] is not None:
                r, count = ref["dw" + n], d[n].shape[0] * d[n].shape[1] * d[n].shape[2]
                size = (count ** 0.5 + 1) * 4  # of a sum of that many terms of about one
                m.check_each("dw" + n, got["dw" + n], r, 1e-5 * size)
            else:
                assert got["dw" + n] is None


QK = [(1, 1, 1, 1, 64, 64), (2, 5, 4, 2, 128, 128), (1, 130, 3, 1, 64, 32), (3, 17, 5, 5, 32, 32), (2, 33, 2, 0, 80, 40),
      (1, 9, 7, 3, 256, 256), (2, 20, 3, 2, 8, 8), (2, 11, 2, 1, 96, 0), (1, 40, 1, 6, 240, 16), (40, 1, 16, 4, 128, 64),
      (1, 700, 12, 4, 64, 64), (2, 3, 100, 1, 72, 24)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", QK)
def test_qk_norm(B, T, Hq, Hk, D, R, dtype, interleaved):
    d = m.qk_inputs(B, T, Hq, Hk, D, R, dtype, interleaved, seed=B + T + D, positions=T % 2 == 1)
    _qk_check(_qk_run(_views(d), _qk_table(d)), m.qk_ref(d), d)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_norm_without_weights(dtype):
    d = m.qk_inputs(2, 30, 4, 2, 64, 64, dtype, seed=31)
    d["wk"] = None
    _qk_check(_qk_run(_views(d), _qk_table(d)), m.qk_ref(d), d)
    d["wq"] = None
    _qk_check(_qk_run(_views(d), _qk_table(d), eps=0.1), m.qk_ref(d, eps=0.1), d)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("how", ["odd start", "odd stride", "two elements", "broadcast heads", "heads outside", "shared positions"])
def test_qk_norm_strides(how, interleaved, dtype):
    B, T, H, D = 2, 21, 3, 64
    d = m.qk_inputs(B, T, H, H, D, 32, dtype, interleaved, seed=32)
    gen = torch.Generator().manual_seed(33)
    n = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
    if how == "odd start":
        d["q"] = n(B, T, H, D + 1)[..., 1:]
        d["grad_k"] = n(B, T, H, D + 1)[..., 1:]
    elif how == "odd stride":
        d["k"], d["grad_q"] = n(B, T, H, D + 1)[..., :-1], n(B, T, H * D + 1)[..., 1:].unflatten(-1, (H, D))
    elif how == "two elements":
        d["q"] = n(B, T, H, D + 2)[..., 2:]
    elif how == "broadcast heads":
        d["k"], d["grad_q"] = d["k"][:, :, :1].expand(B, T, H, D), d["grad_q"][:1, :1].expand(B, T, H, D)
    elif how == "heads outside":  # [B,H,T,D] in memory
        d["q"], d["grad_k"] = n(B, H, T, D).transpose(1, 2), n(B, H, T, D).transpose(1, 2)
    else:
        d["at"] = d["at"][:1].expand(B, T)
    _qk_check(_qk_run(_views(d), _qk_table(d)), m.qk_ref(d), d)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_norm_one_token(dtype):
    d = m.qk_inputs(9, 1, 4, 2, 64, 64, dtype, seed=34)
    c, ref = _views(d), m.qk_ref(d)
    one = {**c, **{n: c[n][:, 0] for n in ("q", "k", "grad_q", "grad_k", "at")}}
    got = _qk_run(one, _qk_table(d))
    _qk_check({n: x.unsqueeze(1) if x.dim() == 3 else x for n, x in got.items()}, ref, d)
    # without positions: the first
    got = _qk_run({**one, "at": None}, _qk_table(d), bwd=False)
    d["at"] = torch.zeros(9, 1, dtype=torch.int32)
    _qk_check({n: x.unsqueeze(1) for n, x in got.items()}, m.qk_ref(d, grads=False), d)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_norm_empty_rows(dtype):
    # positions outside the table: zeros, also for the gradients, whatever lies there
    d = m.qk_inputs(2, 40, 3, 2, 64, 64, dtype, seed=35)
    gen = torch.Generator().manual_seed(36)
    off = torch.rand(2, 40, generator=gen) < 0.4
    off[1] = True
    d["at"][off] = torch.tensor([-1, d["rows"], 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)[torch.randint(4, (int(off.sum()),), generator=gen)]
    ref = m.qk_ref(d)
    # what lies in empty rows does not matter, and is no part of the references' sums
    for n in ("q", "k", "grad_q", "grad_k"):
        d[n] = d[n].clone()
        d[n][off] = torch.nan
    got = _qk_run(_views(d), _qk_table(d))
    for n in ("q", "k"):
        ref["d" + n] = torch.where(off[:, :, None, None], 0.0, ref["d" + n])
        assert not got[n].cpu()[off].any() and not got["d" + n].cpu()[off].any()
    _qk_check(got, ref, d)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_norm_non_finite_stays_in_its_head(dtype):
    d = m.qk_inputs(1, 12, 4, 2, 64, 64, dtype, seed=37)
    clean = m.qk_ref(d)
    d["q"] = d["q"].clone()
    d["q"][0, 5, 2, 9], d["q"][0, 7, 1, 3] = torch.nan, torch.inf
    got = _qk_run(_views(d), _qk_table(d))
    for n in ("q", "dq"):
        g, r = got[n].cpu().clone(), clean[n].clone()
        assert torch.isnan(g[0, 5, 2]).all()
        for t, h in ((5, 2), (7, 1)):
            g[0, t, h], r[0, t, h] = 0, 0
        _ = m.check_each(n, g, r, 100 * U * 16 * r.abs().amax())
    _qk_check({**got, "q": clean["q"].to(dtype), "dq": clean["dq"].to(dtype), "dwq": clean["dwq"].to(dtype)}, clean, d)
    assert torch.isnan(got["dwq"]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_qk_norm_far_positions(dtype):
    d = m.qk_inputs(1, 8, 2, 1, 128, 128, dtype, rows=200000, seed=38)
    d["at"] = torch.tensor([[0, 1, 99999, 131071, 199999, 150000, 65536, 2]], dtype=torch.int32)
    _qk_check(_qk_run(_views(d), _qk_table(d)), m.qk_ref(d), d)


def test_qk_norm_small_and_large_values():
    # squares that underflow beside eps, and heads of zeros; large ones
    for scale in (0.0, 1e-25, 1e-3, 1e15):
        d = m.qk_inputs(1, 5, 2, 1, 64, 64, F32, seed=39)
        d["q"] = d["q"] * scale
        got, ref = _qk_run(_views(d), _qk_table(d), bwd=False), m.qk_ref(d, grads=False)
        _qk_check(got, ref, d)


@pytest.mark.parametrize("shape", [(0, 4, 2, 2), (2, 0, 2, 2), (2, 4, 0, 0)])
def test_qk_norm_empty(shape):
    B, T, Hq, Hk = shape
    q, k = torch.zeros(B, T, Hq, 64, device="cuda"), torch.zeros(B, T, Hk, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    yq, yk = api.qk_norm_fwd(q, k, w, w)
    assert yq.shape == q.shape and yk.shape == k.shape
    dq, dk, dwq, dwk = api.qk_norm_bwd(q, k, w, w, q, k)
    assert not dwq.any() and not dwk.any() and dq.shape == q.shape


def test_qk_norm_gradients_through_autograd():
    d = m.qk_inputs(2, 30, 4, 2, 64, 32, seed=40)
    c, table = _views(d), _qk_table(d)
    leaves = [c[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk")]
    q, k = api.qk_norm(*leaves, table, c["at"])
    ((q * c["grad_q"]).sum() + (k * c["grad_k"]).sum()).backward()
    _qk_check({"q": q, "k": k, **{n: x.grad for n, x in zip(("dq", "dk", "dwq", "dwk"), leaves)}}, m.qk_ref(d), d)
    # one of the two alone
    leaves = [x.detach().requires_grad_() for x in leaves]
    q, k = api.qk_norm(*leaves, table, c["at"])
    (k * c["grad_k"]).sum().backward()
    assert not leaves[0].grad.any() and not leaves[2].grad.any() and leaves[1].grad.any()


# ---------------------------------------------------------------- embedding
def _embed_check(d, V, scale, got=None):
    c = cuda(d)
    dW = api.embedding_bwd(c["tokens"], c["grad"], V, scale) if got is None else got
    ref, mag, count = m.embed_grad_ref(d["tokens"], d["grad"], V, scale)
    m.check_each("dW", dW, ref, (count + 3) * U * mag)
    seen = torch.zeros(V, dtype=torch.bool)
    t = d["tokens"].flatten().long()
    seen[t[(t >= 0) & (t < V)]] = True
    assert not dW.cpu()[~seen].any()
    return dW


EMBED = [(1, 1, 1), (1, 10, 8), (5, 3, 33), (33, 100, 64), (1000, 977, 257), (4097, 50, 128), (3000, 40000, 40),
         (20000, 300, 16), (257, 70000, 8), (513, 2, 2056)]


@pytest.mark.parametrize("kind", [torch.int64, torch.int32])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", EMBED)
def test_embedding(N, V, D, dtype, kind):
    d = m.embed_inputs(N, V, D, dtype, kind, seed=N + V)
    scale = D ** 0.5
    c = cuda(d)
    x = api.embedding_fwd(c["tokens"], c["W"], scale)
    assert torch.equal(x.cpu(), (d["W"].float()[d["tokens"].long()] * torch.tensor(scale, dtype=F32)).to(dtype))
    _embed_check(d, V, scale)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,V,D", [(3000, 64, 72), (9000, 5000, 8), (70, 3, 512), (40000, 100000, 24)])
def test_embedding_few_words(N, V, D, dtype):
    # all of three words, and all of one: long sums, that a single row must not make slow or wrong
    d = m.embed_inputs(N, V, D, dtype, seed=41, few=True)
    _embed_check(d, V, 1.0)
    d["tokens"] = torch.full((N,), V - 1)
    _embed_check(d, V, 0.5)
    # ... in blocks, and each in its turn
    d["tokens"] = torch.arange(N) * V // N
    _embed_check(d, V, 1.0)
    d["tokens"] = torch.arange(N) % V
    _embed_check(d, V, 1.0)


@pytest.mark.parametrize("kind", [torch.int64, torch.int32])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_empty_rows(dtype, kind):
    N, V, D = 500, 60, 48
    d = m.embed_inputs(N, V, D, dtype, kind, seed=42)
    gen = torch.Generator().manual_seed(43)
    off = torch.rand(N, generator=gen) < 0.3
    bad = [-1, V, -2 ** 31, 2 ** 31 - 1] + ([2 ** 32 + 3, -2 ** 63, 2 ** 63 - 1] if kind == torch.int64 else [])
    d["tokens"][off] = torch.tensor(bad, dtype=kind)[torch.randint(len(bad), (int(off.sum()),), generator=gen)]
    d["grad"][off] = torch.nan  # not looked at
    c = cuda(d)
    x = api.embedding_fwd(c["tokens"], c["W"])
    want = d["W"][d["tokens"].long().clamp(0, V - 1)]
    want[off] = 0
    assert torch.equal(x.cpu(), want)
    _embed_check(d, V, 1.0)
    d["tokens"][:] = -1
    assert not api.embedding_bwd(d["tokens"].cuda(), c["grad"], V).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_embedding_strides_and_alignment(dtype):
    N, V, D = 300, 90, 64
    d = m.embed_inputs(N, V, D, dtype, seed=44)
    gen = torch.Generator().manual_seed(45)
    for off, width in ((1, D + 1), (0, D + 1), (0, 2 * D), (4, D + 8)):
        big = torch.randn(N, width, generator=gen).to(dtype)
        d["grad"] = big[:, off:off + D]
        c = _views({"tokens": d["tokens"], "grad": d["grad"]})
        _embed_check(d, V, 2.0, api.embedding_bwd(c["tokens"], c["grad"], V, 2.0))
    d["grad"] = d["grad"][:1].expand(N, D)
    _embed_check(d, V, 1.0, api.embedding_bwd(c["tokens"], c["grad"][:1].expand(N, D), V))
    # a table and tokens that start anywhere
    W = torch.randn(V * D + 1, generator=gen).to(dtype)[1:].view(V, D)
    t = torch.cat([d["tokens"][:1], d["tokens"]])
    c = _views({"W": W, "t": t[1:]})
    assert torch.equal(api.embedding_fwd(c["t"], c["W"]).cpu(), W[d["tokens"]])


def test_embedding_repeats_its_bits_and_shapes():
    d = cuda(m.embed_inputs(6000, 500, 136, seed=46))
    a, c = (api.embedding_bwd(d["tokens"], d["grad"], 500) for _ in range(2))
    assert torch.equal(a, c)
    t = d["tokens"].view(6, 1000)
    assert api.embedding_fwd(t, d["W"]).shape == (6, 1000, 136)
    assert torch.equal(api.embedding_bwd(t, d["grad"].view(6, 1000, 136), 500), a)
    assert api.embedding_fwd(t[0, 0], d["W"]).shape == (136,)
    none = torch.zeros(0, 3, dtype=torch.int64, device="cuda")
    assert api.embedding_fwd(none, d["W"]).shape == (0, 3, 136)
    assert not api.embedding_bwd(none, torch.zeros(0, 3, 136, device="cuda"), 500).any()


def test_embedding_non_finite_stays_in_its_row():
    d = m.embed_inputs(2000, 40, 32, seed=47)
    d["grad"][700, 5], d["grad"][900, 6] = torch.nan, torch.inf
    dW = api.embedding_bwd(d["tokens"].cuda(), d["grad"].cuda(), 40).cpu()
    clean = d["grad"].clone()
    clean[700, 5] = clean[900, 6] = 0
    ref, mag, count = m.embed_grad_ref(d["tokens"], clean, 40, 1.0)
    v, w = d["tokens"][700], d["tokens"][900]
    assert torch.isnan(dW[v, 5]) and dW[w, 6] == torch.inf
    dW[v, 5], dW[w, 6] = ref[v, 5], ref[w, 6]
    m.check_each("dW", dW, ref, (count + 3) * U * mag)


def test_embedding_gradient_through_autograd():
    d = cuda(m.embed_inputs(60, 30, 24, seed=48))
    W = d["W"].clone().requires_grad_()
    t = d["tokens"].view(6, 10)[:, :-1]  # not contiguous
    (api.embedding(t, W, 3.0) * d["grad"].view(6, 10, 24)[:, :-1]).sum().backward()
    ref, mag, count = m.embed_grad_ref(t.cpu(), d["grad"].view(6, 10, 24)[:, :-1].cpu(), 30, 3.0)
    m.check_each("dW", W.grad, ref, (count + 3) * U * mag)
    W.grad = None
    api.embedding(t, W).sum().backward()
    assert torch.equal(W.grad[:, 0].cpu(), torch.bincount(t.flatten().cpu(), minlength=30).float())


# ---------------------------------------------------------------- together
def _layer(tokens, W, wn, wqk, wq, wk, wg, norm, table):
    """Embedding, norm, queries and keys normed and turned, linear attention, then the gated recurrence."""
    x = api.embedding(tokens, W, 2.0)
    y = api.rms_norm(x, wn)
    q, k, v = (y @ wqk).unflatten(-1, (4, 64)).split([1, 1, 2], 2)
    q, k = api.qk_norm(q, k, wq, wk, table)
    g = torch.full((*tokens.shape, 2), -0.1, device=W.device)
    o, _ = api.linear_attention(q, k, v, g)
    h, _ = api.gated_scan(*(o.flatten(-2) @ wg).split(128, -1))
    return (h.float() * norm).sum()


def _layer_args(dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(50)
    n = lambda *s: (torch.randn(s, generator=gen, device="cuda") * 0.3).to(dtype)  # noqa: E731
    tokens = torch.randint(0, 50, (2, 130), generator=gen, device="cuda")
    return tokens, [n(50, 96), n(96) + 1, n(96, 256), n(64) + 1, n(64) + 1, n(128, 256)], n(2, 130, 128).float(), \
        api.rotary_table(130, 64)


def test_a_run_of_them_together():
    tokens, leaves, norm, table = _layer_args()
    leaves = [x.requires_grad_() for x in leaves]
    loss = _layer(tokens, *leaves, norm, table)
    grads = torch.autograd.grad(loss, leaves)
    # the same in 64 bits on the CPU, by torch's own differentiation
    W, wn, wqk, wq, wk, wg = x = [t.detach().cpu().double().requires_grad_() for t in leaves]
    t = tokens.cpu()
    e = 2 * W[t]
    y = e / torch.sqrt((e * e).mean(-1, keepdim=True) + 1e-6) * wn
    q, k, v = (y @ wqk).unflatten(-1, (4, 64)).split([1, 1, 2], 2)
    d = {"R": 64, "rows": 130, "interleaved": False}
    at = torch.arange(130).expand(2, 130)
    q, k = m.qk_forward64(q, wq, at, d, 1e-6), m.qk_forward64(k, wk, at, d, 1e-6)
    S, os = torch.zeros(2, 2, 64, 64, dtype=torch.float64), []
    for i in range(130):
        S = 0.9048374180359595 * S + k[:, i, :, :, None] * v[:, i, :, None, :]
        os.append((S * q[:, i, :, :, None]).sum(2) / 8)
    gate, value = (torch.stack(os, 1).flatten(-2) @ wg).split(128, -1)
    c = torch.where(value >= 0, value + 0.5, torch.sigmoid(value))
    h, hs = torch.zeros(2, 128, dtype=torch.float64), []
    for i in range(130):
        z = torch.sigmoid(gate[:, i])
        h = (1 - z) * h + z * c[:, i]
        hs.append(h)
    want = (torch.stack(hs, 1) * norm.cpu().double()).sum()
    ref = torch.autograd.grad(want, x)
    # g is -0.1 in fp32: exp(-0.1) differs by 1.5e-9 of itself; fp32's errors of the chain: 1e-5 of each norm
    for n, a, r in zip(("W", "wn", "wqk", "wq", "wk", "wg"), grads, ref):
        e = ((a.cpu().double() - r).norm() / r.norm()).item()
        assert e <= 5e-5, (n, e)


def test_captured_and_replayed_with_new_inputs():
    # forward and backward entry points in one graph; replayed on other inputs in the same memory
    d = _views(m.gated_inputs(2, 300, 64, BF16, seed=51))
    e = m.qk_inputs(2, 30, 4, 2, 64, 64, BF16, seed=52)
    f = cuda(m.embed_inputs(700, 90, 64, seed=53))
    table, c = _qk_table(e), _views(e)

    def run():
        return [*_gated_run(d).values(), *_qk_run(c, table).values(), api.embedding_fwd(f["tokens"], f["W"]),
                api.embedding_bwd(f["tokens"], f["grad"], 90)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    gen = torch.Generator(device="cuda").manual_seed(54)
    for _ in range(2):
        for x in (d["gate"], d["value"], d["grad_h"], c["q"], c["k"], f["W"], f["grad"]):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        f["tokens"].copy_(torch.randint(0, 90, (700,), generator=gen, device="cuda"))
        graph.replay()
        for a, w in zip(held, run()):
            assert torch.equal(a, w)
    b.mgs_check()


@pytest.mark.parametrize("address", [False, True])
def test_on_a_named_stream(address):
    # two calls at once, on a stream of their own beside the current one
    d = [_views(m.gated_inputs(2, 500, 64, BF16, seed=55 + i)) for i in range(2)]
    c = [_views(m.qk_inputs(2, 60, 4, 2, 64, 64, BF16, seed=57 + i)) for i in range(2)]
    f = [cuda(m.embed_inputs(2500, 80, 64, seed=59 + i)) for i in range(2)]
    table = api.rotary_table(185, 64)

    def run(i, s=None):
        return [*_gated_run(d[i], stream=s).values(), *_qk_run(c[i], table, stream=s).values(),
                api.embedding_fwd(f[i]["tokens"], f[i]["W"], stream=s), api.embedding_bwd(f[i]["tokens"], f[i]["grad"], 80, stream=s)]

    want = [run(0), run(1)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda._sleep(20_000_000)  # some milliseconds on the current stream
    for _ in range(3):
        got.append([run(i, s.cuda_stream if address else s) for i, s in enumerate(side)])
    torch.full((1 << 20,), 9.0, device="cuda")
    for s in side:
        b.mgs_check(s)
    torch.cuda.synchronize()
    for g in got:
        for i in range(2):
            for a, w in zip(g[i], want[i]):
                assert torch.equal(a, w)


# ---------------------------------------------------------------- sizes and offsets past 32 bits
def _far(shape, dtype, apart, gen):
    """A tensor whose batch rows lie `apart` elements from each other."""
    buf = torch.empty((shape[0] - 1) * apart + shape[1:].numel(), dtype=dtype, device="cuda")
    t = buf.as_strided(shape, (apart, *torch.empty(shape[1:]).stride()))
    return t.copy_(torch.randn(shape, generator=gen, device="cuda"))


def test_offsets_past_32_bits():
    gen = torch.Generator(device="cuda").manual_seed(61)
    apart = (1 << 31) + 64
    # rows of inputs 2^31 elements apart
    gate, value, gh = (_far(torch.Size((2, 70, 64)), BF16, apart, gen) for _ in range(3))
    near = [x.contiguous() for x in (gate, value, gh)]
    a, w = api.gated_scan_fwd(gate, value, want_carries=True), api.gated_scan_fwd(*near[:2], want_carries=True)
    assert all(torch.equal(x, y) for x, y in zip(a, w))
    for x, y in zip(api.gated_scan_bwd(gate, value, a[2], gh), api.gated_scan_bwd(*near[:2], w[2], near[2])):
        assert torch.equal(x, y)
    del gate, value, gh
    q, gq = (_far(torch.Size((2, 9, 2, 64)), BF16, apart, gen) for _ in range(2))
    table, c, gc = api.rotary_table(9, 64), q.contiguous(), gq.contiguous()
    for x, y in zip(api.qk_norm_fwd(q, q, table=table), api.qk_norm_fwd(c, c, table=table)):
        assert torch.equal(x, y)
    for x, y in zip(api.qk_norm_bwd(q, q, None, None, gq, gq, table)[:2], api.qk_norm_bwd(c, c, None, None, gc, gc, table)[:2]):
        assert torch.equal(x, y)
    del q, gq
    # a cache and a table of more than 2^31 elements
    N, D = 530000, 4096
    state = torch.empty(N, D, device="cuda")
    slots = torch.tensor([N - 1, 3, N - 2], dtype=torch.int32, device="cuda")
    state[slots.long()] = torch.randn(3, D, generator=gen, device="cuda")
    small = state[slots.long()].clone()
    k, v = torch.randn(3, D, generator=gen, device="cuda"), torch.randn(3, D, generator=gen, device="cuda")
    assert torch.equal(api.gated_scan_step(k, v, state, slots), api.gated_scan_step(k, v, small))
    assert torch.equal(state[slots.long()], small)
    W = state  # (the same memory as a table)
    tokens = torch.tensor([N - 1, 0, N - 2, N - 1, 3], device="cuda")
    assert torch.equal(api.embedding_fwd(tokens, W), W[tokens])
    del W, state
    g = torch.randn(5, D, generator=gen, device="cuda").to(BF16)
    dW = api.embedding_bwd(tokens, g, N)
    assert torch.equal(dW[N - 1], (g[0].float() + g[3].float()).to(BF16)) and torch.equal(dW[N - 2], g[2])
    assert torch.equal(dW[3], g[4]) and dW.count_nonzero().item() == sum(dW[i].count_nonzero().item() for i in (0, 3, N - 2, N - 1))


def test_large_vocabulary():
    # more rows than the blocks mark at a time
    V, N = 6_000_000, 5000
    gen = torch.Generator(device="cuda").manual_seed(62)
    tokens = torch.randint(0, V, (N,), generator=gen, device="cuda")
    tokens[:700] = V - 1
    g = torch.randn(N, 8, generator=gen, device="cuda")
    dW = api.embedding_bwd(tokens, g, V)
    ref = torch.zeros(V, 8, dtype=torch.float64, device="cuda").index_add_(0, tokens, g.double())
    mag = torch.zeros(V, 8, dtype=torch.float64, device="cuda").index_add_(0, tokens, g.double().abs())
    assert ((dW.double() - ref).abs() <= 703 * U * mag).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_tokens_of_one_width(dtype):
    # more places than a block keeps in registers, odd rows; and bf16 rows that start anywhere
    d = m.embed_inputs(70001, 3000, 33, dtype, seed=63)
    _embed_check(d, 3000, 1.0)


@pytest.mark.parametrize("B,T,D", [(70000, 3, 2), (1, 100001, 1), (3, 64, 5000)])
def test_gated_many_of_one_dimension(B, T, D):
    # 400 u of the largest covers memories of 100 steps whatever the length; one channel's reference on the GPU
    d = m.gated_inputs(B, T, D, seed=64, shift=1.0)
    if T < 1000:
        _gated_check(_gated_run(_views(d)), m.gated_ref(d))
        return
    c = _views(d)
    got = _gated_run(c)
    whole = m.gated_ref({**d, "gate": d["gate"][:, -3000:], "value": d["value"][:, -3000:], "grad_h": d["grad_h"][:, -3000:],
                         "h0": got["h"][:, -3001].cpu()})
    for n in ("h", "dgate", "dvalue"):  # the end, from the state that the call itself has there
        m.check_each(n, got[n][:, -3000:], whole[n], 400 * U * whole[n].abs().amax())


def test_gradients_of_some_leaves():
    d = _views(m.gated_inputs(2, 40, 16, seed=65))
    gate = d["gate"].clone().requires_grad_()
    h, hT = api.gated_scan(gate, d["value"])
    hT.sum().backward()
    ref = m.gated_ref({**{n: (x.cpu() if isinstance(x, torch.Tensor) else x) for n, x in d.items()}, "h0": None,
                       "grad_h": torch.zeros(2, 40, 16), "grad_hT": torch.ones(2, 16)})
    m.check_each("dgate", gate.grad, ref["dgate"], 400 * U * ref["dgate"].abs().amax(1, keepdim=True))
    with torch.no_grad():
        assert not api.gated_scan(gate, d["value"])[0].requires_grad
