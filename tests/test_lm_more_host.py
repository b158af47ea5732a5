"""Checks of the gated recurrence, the norm of queries and keys and the embedding
that need no GPU: the references of their tests against differences, the refusals
of the C ABI (fake, never-dereferenced addresses) and of the tensor functions, and
what those do around a call of the library."""
import contextlib

import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api
from scan_linear_recurrences_gb300.build import build

from . import _lm_more as m

FAKE = 1 << 40
OK, INVALID, UNSUPPORTED, WORKSPACE = b.MGS_OK, b.MGS_ERR_INVALID_ARG, b.MGS_ERR_UNSUPPORTED, b.MGS_ERR_WORKSPACE
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def _st(fn, *args):
    try:
        fn(*args, stream=0)
        return OK
    except b.MGSError as e:
        return e.status


def _differences(loss, x, names, grads, gen, tol=1e-7):
    # central differences in 64 bits: truncation eps^2, rounding 1e-16 / eps
    for n in names:
        u, eps = torch.randn(x[n].shape, generator=gen, dtype=torch.float64), 1e-5
        hi, lo = loss({**x, n: x[n] + eps * u}), loss({**x, n: x[n] - eps * u})
        want = (grads[n] * u).sum()
        assert abs((hi - lo) / (2 * eps) - want) <= tol * (1 + abs(want)), n


@pytest.mark.parametrize("positive", [False, True])
def test_gated_reference_gradients_against_differences(positive):
    d = m.gated_inputs(2, 6, 3, seed=3, positive=positive)
    x = {n: (t.double() if isinstance(t, torch.Tensor) else t) for n, t in d.items()}
    ref = m.gated_ref(x)

    def loss(x):
        o = m.gated_ref(x, grads=False)
        return (o["h"] * x["grad_h"]).sum() + (o["h_T"] * x["grad_hT"]).sum()

    _differences(loss, x, ("gate", "value", "h0"), {"gate": ref["dgate"], "value": ref["dvalue"], "h0": ref["dh0"]},
                 torch.Generator().manual_seed(4))


@pytest.mark.parametrize("interleaved,R", [(False, 16), (True, 8), (False, 0)])
def test_qk_reference_gradients_against_differences(interleaved, R):
    d = m.qk_inputs(2, 3, 2, 1, 16, R, interleaved=interleaved, seed=5)
    ref = m.qk_ref(d)
    x = {n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for n, t in d.items()}

    def loss(x):
        o = m.qk_ref(x, grads=False)
        return (o["q"] * x["grad_q"]).sum() + (o["k"] * x["grad_k"]).sum()

    _differences(loss, x, ("q", "k", "wq", "wk"), {n: ref["d" + n] for n in ("q", "k", "wq", "wk")},
                 torch.Generator().manual_seed(6))


def test_rotary_table():
    t = api.rotary_table(70001, 16, base=500.0, device="cpu")
    a = m.angles(70001, 16, 500.0)
    assert t.shape == (70001, 16) and t.dtype == F32
    assert (t[:, :8].double() - a.cos()).abs().max() <= 2.0 ** -24 and (t[:, 8:].double() - a.sin()).abs().max() <= 2.0 ** -24
    assert api.rotary_table(0, 8, device="cpu").shape == (0, 8)
    with pytest.raises(ValueError, match="even"):
        api.rotary_table(4, 7, device="cpu")


# ---------------------------------------------------------------- refusals of the C ABI
def _gated(B=2, T=100, D=64, dtype=b.MGS_BF16, ks=None, vs=None, gs=None):
    s = (T * D, D)
    return b.mgs_gated_shape(B, T, D, dtype, 1, ks or s, vs or s, gs or s)


def test_gated_refusals():
    k, v, h0, h, hT, c = (FAKE + i * (1 << 30) for i in range(6))
    f = b.mgs_gated_scan_fwd
    assert _st(f, None, k, v, h0, h, hT, c) == INVALID
    assert _st(f, _gated(B=-1), k, v, h0, h, hT, c) == INVALID
    assert _st(f, _gated(dtype=7), k, v, h0, h, hT, c) == UNSUPPORTED
    assert _st(f, _gated(ks=(-64, 64)), k, v, h0, h, hT, c) == UNSUPPORTED
    assert _st(f, _gated(B=1 << 31, T=1 << 30, D=8), k, v, h0, h, hT, c) == INVALID
    assert _st(f, _gated(B=2, T=2, ks=(1 << 62, 64)), k, v, h0, h, hT, c) == UNSUPPORTED
    assert _st(f, _gated(), None, v, h0, h, hT, c) == INVALID
    assert _st(f, _gated(), k, v, h0, None, hT, c) == INVALID
    assert _st(f, _gated(), k + 1, v, h0, h, hT, c) == UNSUPPORTED
    assert _st(f, _gated(), k, v, h0 + 2, h, hT, c) == UNSUPPORTED
    assert _st(f, _gated(), k, v, h0, h, hT, c + 2) == UNSUPPORTED
    for outs in ((k, hT, c), (h, h0, c), (h, hT, h0), (h, h + 64, c), (h, hT, v + 128)):  # over inputs or each other
        assert _st(f, _gated(), k, v, h0, *outs) == INVALID
    # (outputs in the gaps of a strided input count as over it)
    assert _st(f, _gated(ks=(12800, 128)), k, v, h0, k + 128, hT, c) == INVALID
    assert _st(f, _gated(B=0), None, None, None, None, None, None) == OK
    assert _st(f, _gated(D=0), None, None, None, None, None, None) == OK
    assert _st(f, _gated(T=0), None, None, None, None, None, None) == OK
    gh, ghT, dk, dv, d0 = (FAKE + i * (1 << 30) for i in range(6, 11))
    bwd = b.mgs_gated_scan_bwd
    assert _st(bwd, _gated(), k, v, None, gh, ghT, dk, dv, d0) == INVALID
    assert _st(bwd, _gated(), k, v, c, None, ghT, dk, dv, d0) == INVALID
    assert _st(bwd, _gated(), k, v, c, gh, ghT, None, dv, d0) == INVALID
    assert _st(bwd, _gated(), k, v, c, gh, ghT, gh, dv, d0) == INVALID
    assert _st(bwd, _gated(), k, v, c, gh, ghT, dk, dk, d0) == INVALID
    assert _st(bwd, _gated(), k, v, c, gh, ghT, dk, dv, ghT) == INVALID
    assert _st(bwd, _gated(gs=(-1, 1)), k, v, c, gh, ghT, dk, dv, d0) == UNSUPPORTED
    assert _st(bwd, _gated(), k, v, c, gh + 1, ghT, dk, dv, d0) == UNSUPPORTED
    assert _st(bwd, _gated(T=0), None, None, None, None, ghT, None, None, ghT) == INVALID
    assert _st(bwd, _gated(B=0), None, None, None, None, None, None, None, None) == OK


def test_gated_step_refusals():
    k, v, s, slots, h = (FAKE + i * (1 << 30) for i in range(5))
    f = b.mgs_gated_scan_step
    assert _st(f, _gated(T=2), k, v, s, slots, 8, h) == INVALID
    assert _st(f, None, k, v, s, slots, 8, h) == INVALID
    assert _st(f, _gated(T=1), k, v, s, None, 1, h) == INVALID      # fewer states than sequences
    assert _st(f, _gated(T=1), k, v, s, slots, -1, h) == INVALID
    assert _st(f, _gated(T=1), k, v, None, slots, 8, h) == INVALID
    assert _st(f, _gated(T=1), k, v, s, slots + 2, 8, h) == UNSUPPORTED
    assert _st(f, _gated(T=1), k, v, s, slots, 8, s) == INVALID
    assert _st(f, _gated(T=1), s, v, s, slots, 8, h) == INVALID
    assert _st(f, _gated(T=1), k, v, s, slots, 1 << 60, h) == INVALID
    assert _st(f, _gated(T=1, B=0), None, None, None, None, 0, None) == OK


def _qk(B=2, T=8, Hq=4, Hk=2, rows=16, D=64, dtype=b.MGS_BF16, R=64, qs=None, gs=None, ps=(8, 1)):
    q, k = (T * Hq * D, Hq * D, D), (T * Hk * D, Hk * D, D)
    return b.mgs_qk_norm_shape(B, T, Hq, Hk, rows, D, dtype, R, 0, 1e-6, qs or q, k, gs or q, k, ps)


def test_qk_norm_refusals():
    q, k, wq, wk, tab, pos, yq, yk = (FAKE + i * (1 << 30) for i in range(8))
    f = b.mgs_qk_norm_fwd
    assert _st(f, None, q, k, wq, wk, tab, pos, yq, yk) == INVALID
    assert _st(f, _qk(Hq=-1), q, k, wq, wk, tab, pos, yq, yk) == INVALID
    for bad in ({"D": 60}, {"D": 264}, {"D": 0, "R": 0}, {"R": 72}, {"R": 12}, {"R": -8}, {"dtype": 5}):
        assert _st(f, _qk(**bad), q, k, wq, wk, tab, pos, yq, yk) == UNSUPPORTED, bad
    assert _st(f, _qk(qs=(-1, 64, 64)), q, k, wq, wk, tab, pos, yq, yk) == UNSUPPORTED
    assert _st(f, _qk(ps=(-8, 1)), q, k, wq, wk, tab, pos, yq, yk) == UNSUPPORTED
    assert _st(f, _qk(), q + 1, k, wq, wk, tab, pos, yq, yk) == UNSUPPORTED
    assert _st(f, _qk(), q, k, wq, wk, tab + 8, pos, yq, yk) == UNSUPPORTED
    assert _st(f, _qk(), q, k, wq, wk, tab, pos + 2, yq, yk) == UNSUPPORTED
    assert _st(f, _qk(), None, k, wq, wk, tab, pos, yq, yk) == INVALID
    assert _st(f, _qk(), q, k, wq, wk, None, pos, yq, yk) == INVALID       # rotated elements without a table
    assert _st(f, _qk(R=0), q, k, wq, wk, tab, None, yq, yk) == INVALID    # a table without rotated elements
    assert _st(f, _qk(R=0), q, k, wq, wk, None, pos, yq, yk) == INVALID    # positions without a table
    assert _st(f, _qk(rows=7), q, k, wq, wk, tab, None, yq, yk) == INVALID  # fewer rows than steps
    for outs in ((q, yk), (yq, k + 64), (yq, yq), (tab, yk), (wq, yk), (yq, pos)):
        assert _st(f, _qk(), q, k, wq, wk, tab, pos, *outs) == INVALID
    assert _st(f, _qk(B=0), None, None, None, None, None, None, None, None) == OK
    bwd = b.mgs_qk_norm_bwd
    gq, gk, dq, dk, dwq, dwk, ws = (FAKE + i * (1 << 30) for i in range(8, 15))
    n = b.mgs_qk_norm_bwd_workspace_size(_qk())
    assert n > 0 and b.mgs_qk_norm_bwd_workspace_size(_qk(D=60)) == 0 and b.mgs_qk_norm_bwd_workspace_size(_qk(B=0)) == 0
    ins = (q, k, wq, wk, gq, gk, tab, pos)
    assert _st(bwd, _qk(), *ins, dq, dk, dwq, dwk) == WORKSPACE
    assert _st(bwd, _qk(), *ins, dq, dk, dwq, dwk, ws, n - 1) == WORKSPACE
    assert _st(bwd, _qk(), *ins, dq, dk, dwq, dwk, ws + 16, n) == WORKSPACE
    assert _st(bwd, _qk(), *ins, dq, None, dwq, dwk, ws, n) == INVALID
    assert _st(bwd, _qk(), q, k, wq, wk, None, gk, tab, pos, dq, dk, dwq, dwk, ws, n) == INVALID
    for outs in ((gq, dk, dwq, dwk), (dq, dk, dwq, dwq), (dq, dk, wq, dwk), (dq, dk, ws, dwk)):
        assert _st(bwd, _qk(), *ins, *outs, ws, n) == INVALID
    assert _st(bwd, _qk(gs=(-1, 1, 64)), *ins, dq, dk, dwq, dwk, ws, n) == UNSUPPORTED


def test_embedding_refusals():
    t, w, o = (FAKE + i * (1 << 30) for i in range(3))
    f = b.mgs_embedding_fwd
    assert _st(f, t, b.MGS_I64, w, 1.0, o, -1, 10, 8, b.MGS_F32) == INVALID
    assert _st(f, t, 0, w, 1.0, o, 4, 10, 8, b.MGS_F32) == UNSUPPORTED
    assert _st(f, t, b.MGS_I64, w, 1.0, o, 4, 10, 8, 9) == UNSUPPORTED
    assert _st(f, t + 4, b.MGS_I64, w, 1.0, o, 4, 10, 8, b.MGS_F32) == UNSUPPORTED
    assert _st(f, t, b.MGS_I64, w + 2, 1.0, o, 4, 10, 8, b.MGS_F32) == UNSUPPORTED
    assert _st(f, None, b.MGS_I64, w, 1.0, o, 4, 10, 8, b.MGS_F32) == INVALID
    assert _st(f, t, b.MGS_I64, None, 1.0, o, 4, 10, 8, b.MGS_F32) == INVALID
    assert _st(f, t, b.MGS_I64, w, 1.0, w + 32, 4, 10, 8, b.MGS_F32) == INVALID
    assert _st(f, t, b.MGS_I64, w, 1.0, t, 4, 10, 8, b.MGS_F32) == INVALID
    assert _st(f, t, b.MGS_I64, w, 1.0, o, 1 << 62, 10, 8, b.MGS_F32) == INVALID
    assert _st(f, None, b.MGS_I64, None, 1.0, None, 0, 10, 8, b.MGS_F32) == OK
    assert _st(f, None, b.MGS_I64, None, 1.0, None, 5, 10, 0, b.MGS_F32) == OK
    g, dw, ws = (FAKE + i * (1 << 30) for i in range(3, 6))
    bwd, n = b.mgs_embedding_bwd, b.mgs_embedding_bwd_workspace_size(4, 10, 8)
    assert n > 0 and b.mgs_embedding_bwd_workspace_size(-1, 10, 8) == 0 and b.mgs_embedding_bwd_workspace_size(0, 10, 8) == 0
    assert _st(bwd, t, b.MGS_I64, g, 8, 1.0, dw, 4, 10, 8, b.MGS_F32) == WORKSPACE
    assert _st(bwd, t, b.MGS_I64, g, 8, 1.0, dw, 4, 10, 8, b.MGS_F32, ws + 8, n) == WORKSPACE
    assert _st(bwd, t, b.MGS_I64, g, -8, 1.0, dw, 4, 10, 8, b.MGS_F32, ws, n) == UNSUPPORTED
    assert _st(bwd, t, b.MGS_I64, None, 8, 1.0, dw, 4, 10, 8, b.MGS_F32, ws, n) == INVALID
    assert _st(bwd, t, b.MGS_I64, g, 8, 1.0, None, 4, 10, 8, b.MGS_F32, ws, n) == INVALID
    assert _st(bwd, t, b.MGS_I64, g, 8, 1.0, g + 64, 4, 10, 8, b.MGS_F32, ws, n) == INVALID
    assert _st(bwd, t, b.MGS_I64, g, 8, 1.0, dw, 4, 10, 8, b.MGS_F32, dw, n) == INVALID
    assert _st(bwd, t, b.MGS_I32, g, 8, 1.0, dw, 1 << 31, 10, 8, b.MGS_F32, ws, n) == UNSUPPORTED
    assert _st(bwd, None, b.MGS_I64, None, 8, 1.0, None, 4, 0, 8, b.MGS_F32) == OK


# ---------------------------------------------------------------- the tensor functions
def test_tensor_functions_refuse_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        api.gated_scan_fwd(x, x)
    with pytest.raises(ValueError, match=r"\[B,T,D\]"):
        api.gated_scan_fwd(x[0], x[0])
    with pytest.raises(ValueError, match=r"\[B,D\]"):
        api.gated_scan_step(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        api.gated_scan_step(x[0], x[0], x[0])
    with pytest.raises(ValueError, match="CUDA"):
        api.qk_norm_fwd(x[None], x[None])
    with pytest.raises(ValueError, match="Hq"):
        api.qk_norm_fwd(x[0], x[0])
    with pytest.raises(ValueError, match="CUDA"):
        api.embedding_fwd(torch.zeros(3, dtype=torch.int64), x[0])
    with pytest.raises(ValueError, match="CUDA"):
        api.embedding_bwd(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 5)


def test_tensor_functions_refuse(monkeypatch):
    """What is refused once tensors are on the GPU (the check of the device is replaced)."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))

    class Card:
        type, index = "cuda", 0
    x, q, card = torch.zeros(2, 4, 8), torch.zeros(2, 4, 2, 16), Card()
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: card))
    for what, fn in (
            ("float32 or bfloat16", lambda: api.gated_scan_fwd(x.half(), x.half())),
            ("value must be float32", lambda: api.gated_scan_fwd(x, x.bfloat16())),
            ("value has shape", lambda: api.gated_scan_fwd(x, x[:, :3])),
            ("last dimension", lambda: api.gated_scan_fwd(x.transpose(1, 2), x.transpose(1, 2))),
            ("h0 has shape", lambda: api.gated_scan_fwd(x, x, x[:, 0, :4])),
            ("h0 must be float32", lambda: api.gated_scan_fwd(x.bfloat16(), x.bfloat16(), x[:, 0].bfloat16())),
            ("carries has shape", lambda: api.gated_scan_bwd(x, x, torch.zeros(2, 2, 8), x)),
            ("fewer|as many states", lambda: api.gated_scan_step(x[:, 0], x[:, 0], torch.zeros(1, 8))),
            ("slots must be int32", lambda: api.gated_scan_step(x[:, 0], x[:, 0], torch.zeros(3, 8), torch.zeros(2).long())),
            ("state has shape", lambda: api.gated_scan_step(x[:, 0], x[:, 0], torch.zeros(3, 9))),
            ("multiples of 8", lambda: api.qk_norm_fwd(q[..., :12], q[..., :12])),
            ("k has shape", lambda: api.qk_norm_fwd(q, q[:, :3])),
            ("k must be bfloat16", lambda: api.qk_norm_fwd(q.bfloat16(), q)),
            ("q_weight has shape", lambda: api.qk_norm_fwd(q, q, torch.zeros(8))),
            ("rotated elements", lambda: api.qk_norm_fwd(q, q, table=torch.zeros(9, 24))),
            ("rotated elements", lambda: api.qk_norm_fwd(q, q, table=torch.zeros(9, 12))),
            ("need a table of as many rows", lambda: api.qk_norm_fwd(q, q, table=torch.zeros(3, 16))),
            ("without a table", lambda: api.qk_norm_fwd(q, q, positions=torch.zeros(2, 4, dtype=torch.int32))),
            ("positions must be int32", lambda: api.qk_norm_fwd(q, q, table=torch.zeros(9, 16), positions=torch.zeros(2, 4).long())),
            ("positions has shape", lambda: api.qk_norm_fwd(q, q, table=torch.zeros(9, 16), positions=torch.zeros(4, dtype=torch.int32))),
            ("grad_q has shape", lambda: api.qk_norm_bwd(q, q, None, None, q[:, :2], q)),
            ("must be tensors", lambda: api.qk_norm_bwd(q, q, None, None, None, q)),
            ("int32 or int64", lambda: api.embedding_fwd(torch.zeros(3), x[0])),
            (r"\[V,D\]", lambda: api.embedding_fwd(torch.zeros(3).long(), x)),
            ("tokens must be contiguous", lambda: api.embedding_fwd(torch.zeros(3, 2).long().T, x[0])),
            ("grad has shape", lambda: api.embedding_bwd(torch.zeros(3).long(), x[0], 5)),
            ("fixed distance", lambda: api.embedding_bwd(torch.zeros(2, 4).long(), torch.zeros(4, 2, 8).transpose(0, 1), 5)),
    ):
        with pytest.raises(ValueError, match=what):
            fn()


class _Calls:
    """The entry points' calls (replaced), and the streams that were torch's current ones when memory was taken."""

    def __init__(self, monkeypatch):
        self.current, self.scratch, self.calls = ["current"], [], []

        @contextlib.contextmanager
        def on(stream):
            self.current.append(stream)
            yield
            self.current.pop()

        empty = torch.empty

        def new(*a, **k):
            if k.get("dtype") is torch.uint8:
                self.scratch.append(self.current[-1])
            return empty(*a, **k)

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, device=None: ("external", at))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
        monkeypatch.setattr(torch, "empty", new)
        monkeypatch.setattr(api, "_check_typed", lambda *a, **k: None)
        for name in ("gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "qk_norm_fwd", "qk_norm_bwd", "embedding_fwd",
                     "embedding_bwd"):
            monkeypatch.setattr(b, "mgs_" + name, lambda *a, _name=name: self.calls.append((_name, a)))
        monkeypatch.setattr(b, "mgs_qk_norm_bwd_workspace_size", lambda shape: 256)
        monkeypatch.setattr(b, "mgs_embedding_bwd_workspace_size", lambda N, V, D: 256)


@pytest.mark.parametrize("stream,name", [(1234, ("external", 1234)), (0, "default"), ("a torch stream", "a torch stream"),
                                         (None, "current")])
def test_workspace_belongs_to_the_named_stream(monkeypatch, stream, name):
    calls = _Calls(monkeypatch)
    x, q, t = torch.zeros(2, 4, 8), torch.zeros(2, 4, 2, 16), torch.zeros(2, 4).long()
    api.gated_scan_bwd(x, x, x[:, :1], x, stream=stream)
    api.qk_norm_bwd(q, q, None, None, q, q, stream=stream)
    api.embedding_bwd(t, x, 5, stream=stream)
    assert calls.scratch == [name, name] and all(a[-1] is stream for _, a in calls.calls) and len(calls.calls) == 3


def test_states_written_in_place_are_marked_for_autograd(monkeypatch):
    _Calls(monkeypatch)
    x, state, out = torch.zeros(2, 8), torch.zeros(3, 8), torch.zeros(2, 8)
    api.gated_scan_step(x, x, state, out=out)
    assert [t._version for t in (x, state, out)] == [0, 1, 1]


def test_strides_reach_the_library(monkeypatch):
    calls = _Calls(monkeypatch)
    both = torch.zeros(2, 6, 16)
    gate, value = both.split(8, -1)
    api.gated_scan_fwd(gate, value[:, :1].expand(2, 6, 8))
    want = b.mgs_gated_shape(2, 6, 8, b.MGS_F32, 1, (96, 16), (96, 0))
    assert calls.calls[-1][1][0] == want
    q = torch.zeros(2, 3, 32)[:, :2].unflatten(-1, (2, 16))
    at = torch.zeros(2, dtype=torch.int32)
    api.qk_norm_fwd(q[:, 0], q[:, 0, :1], table=torch.zeros(9, 8), positions=at)
    want = b.mgs_qk_norm_shape(2, 1, 2, 1, 9, 16, b.MGS_F32, 8, 0, 1e-6, (96, 0, 16), (96, 0, 16), pos_stride=(1, 0))
    assert calls.calls[-1][1][0] == want
    api.embedding_bwd(torch.zeros(2, 3).long(), torch.zeros(8).expand(2, 3, 8), 5)
    assert calls.calls[-1][1][3] == 0  # the same row for all tokens


def test_second_derivatives_are_refused(monkeypatch):
    monkeypatch.setattr(api, "gated_scan_fwd", lambda k, v, h0, p, want_carries: (k.detach() * v, v.detach()[:, 0], k.detach()))
    monkeypatch.setattr(api, "gated_scan_bwd", lambda k, v, c, gh, ghT, p, need: (gh.detach() * v, gh.detach() * k, None))
    monkeypatch.setattr(api, "qk_norm_fwd", lambda q, k, *a: (q.detach() * 2, k.detach() * 2))
    monkeypatch.setattr(api, "qk_norm_bwd", lambda q, k, wq, wk, gq, gk, *a: (gq.detach() * 2, gk.detach() * 2, None, None))
    monkeypatch.setattr(api, "embedding_fwd", lambda t, w, s: w.detach()[t])
    monkeypatch.setattr(api, "embedding_bwd", lambda t, g, V, s: g.detach().sum(0, keepdim=True).expand(V, -1).clone())
    x = torch.ones(1, 2, 8, requires_grad=True)
    w = torch.ones(4, 8, requires_grad=True)
    for y, leaf in ((api.gated_scan(x, x)[0], x), (api.qk_norm(x[None], x[None])[0], x),
                    (api.embedding(torch.tensor([1, 2]), w), w)):
        d, = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            ((d * d).sum() + (leaf * leaf).sum()).backward()


def test_gradients_that_do_not_arrive_are_zeros(monkeypatch):
    # of two outputs one may go unused: its gradient is one row of zeros, not a tensor of them
    calls = _Calls(monkeypatch)
    x = torch.zeros(2, 4, 8, requires_grad=True)
    h, hT = api.gated_scan(x, x, torch.zeros(2, 8))
    hT.sum().backward()
    shape, *_ = calls.calls[-1][1]
    assert shape == b.mgs_gated_shape(2, 4, 8, b.MGS_F32, 1, (32, 8), (32, 8), (0, 0))
    q = torch.zeros(2, 4, 2, 8, requires_grad=True)
    yq, yk = api.qk_norm(q, q)
    yk.sum().backward()  # an expanded gradient, whose heads are not contiguous: copied
    shape, *_ = calls.calls[-1][1]
    assert shape == b.mgs_qk_norm_shape(2, 4, 2, 2, 0, 8, b.MGS_F32, 0, 0, 1e-6, (64, 16, 8), (64, 16, 8), (0, 0, 0),
                                        (64, 16, 8))


def test_calls_on_another_device_go_there(monkeypatch):
    # the library launches on the current device: a call on another one's tensors makes that one current
    calls = _Calls(monkeypatch)
    there = []

    @contextlib.contextmanager
    def device(d):
        there.append(d)
        yield
        there.append("back")

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "_elsewhere", lambda t: not there or there[-1] == "back")
    x, q, t = torch.zeros(2, 4, 8), torch.zeros(2, 4, 2, 16), torch.zeros(2, 4).long()
    for i, call in enumerate((lambda: api.gated_scan_fwd(x, x), lambda: api.gated_scan_bwd(x, x, x[:, :1], x),
                              lambda: api.gated_scan_step(x[:, 0], x[:, 0], x[:, 1].clone()), lambda: api.qk_norm_fwd(q, q),
                              lambda: api.qk_norm_bwd(q, q, None, None, q, q), lambda: api.embedding_fwd(t, x[0]),
                              lambda: api.embedding_bwd(t, x, 5))):
        call()
        assert there[2 * i:] == [torch.device("cpu"), "back"] and len(calls.calls) == i + 1


def test_differentiable_forms_refuse_what_is_no_tensor():
    # as the plain forms do
    x, w = torch.zeros(2, 4, 8), torch.zeros(4, 8)
    for fn in (lambda: api.gated_scan(None, x), lambda: api.gated_scan([1.0], [2.0]), lambda: api.gated_scan(torch.zeros(()), x),
               lambda: api.qk_norm(None, x), lambda: api.qk_norm(x[None], 3), lambda: api.qk_norm(torch.zeros(()), x),
               lambda: api.embedding([1, 2], w), lambda: api.embedding(torch.zeros(2).long(), None)):
        with pytest.raises((TypeError, ValueError), match="must"):
            fn()


# ---------------------------------------------------------------- the short checks beside the full ones
def _odd(*shape):  # rows of odd starts and distances
    return torch.zeros(*shape[:-1], shape[-1] + 3)[..., 1:-2]


def test_short_checks_make_the_same_call_as_the_full_ones(monkeypatch):
    calls = _Calls(monkeypatch)
    monkeypatch.setattr(api, "_elsewhere", lambda t: False)
    x, h0, q = torch.zeros(2, 70, 2 * 8).split(8, -1), torch.zeros(2, 8), torch.zeros(3, 5, 6, 16).split([4, 2], 2)
    carries, state, slots = torch.zeros(2, 2, 8), torch.zeros(4, 8), torch.zeros(2, dtype=torch.int32)
    table, at, w = torch.zeros(9, 8), torch.zeros(1, 5, dtype=torch.int32).expand(3, 5), torch.zeros(16)
    one, few = [t[:, 1] for t in q], torch.zeros(6, dtype=torch.int32)[::2]
    made = [
        lambda: api.gated_scan_fwd(*x, h0, False),
        lambda: api.gated_scan_fwd(x[0], _odd(2, 70, 8), want_carries=True),
        lambda: api.gated_scan_fwd(x[0].bfloat16(), x[1].bfloat16()[:, :1].expand(2, 70, 8)),
        lambda: api.gated_scan_bwd(*x, carries, _odd(2, 70, 8), h0),
        lambda: api.gated_scan_step(x[0][:, 3], _odd(2, 8), state, slots),
        lambda: api.gated_scan_step(x[0][:, 3], x[1][:, 3], state, positive=False),
        lambda: api.qk_norm_fwd(*q, w, None, table, at, eps=0.5, interleaved=True),
        lambda: api.qk_norm_fwd(*q, None, w, table),
        lambda: api.qk_norm_fwd(*q),
        lambda: api.qk_norm_fwd(*one, w, w, table, few),
        lambda: api.qk_norm_fwd(*one, table=table[:1]),
        lambda: api.qk_norm_fwd(q[0], q[1][:, :, :0]),
        lambda: api.qk_norm_bwd(*q, w, None, _odd(3, 5, 4, 16), q[0][:, :, :1].expand(3, 5, 2, 16), table),
        lambda: api.qk_norm_bwd(*one, None, None, one[0], one[1], table, few),
    ]

    def shapes():
        for fn in made:
            fn()
        return [args[0] for _, args in calls.calls[-len(made):]]

    full = shapes()

    def refused(*a, **k):
        raise AssertionError("the full check ran")

    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    for name in ("_qk_shape_checked", "_gated_step_check"):
        monkeypatch.setattr(api, name, refused)
    monkeypatch.setattr(api, "_inner", refused)
    assert shapes() == full


def test_short_checks_pass_on_what_the_full_ones_refuse(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)

    class Card:
        type, index = "cuda", 0
    card = Card()
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: card))
    monkeypatch.setattr(api, "_elsewhere", lambda t: False)
    x, q, one = torch.zeros(2, 4, 8), torch.zeros(2, 4, 2, 16), torch.zeros(2, 2, 16)
    state, slots, table, w = torch.zeros(3, 8), torch.zeros(2, dtype=torch.int32), torch.zeros(9, 16), torch.zeros(16)
    at = torch.zeros(2, 4, dtype=torch.int32)
    for i, fn in enumerate((
            lambda: api.gated_scan_fwd(x.half(), x.half()), lambda: api.gated_scan_fwd(x, x.bfloat16()),
            lambda: api.gated_scan_fwd(x, x[:, :3]), lambda: api.gated_scan_fwd(x.transpose(1, 2), x.transpose(1, 2)),
            lambda: api.gated_scan_fwd(x, x.transpose(0, 1).transpose(1, 2)), lambda: api.gated_scan_fwd(x[0], x[0]),
            lambda: api.gated_scan_bwd(x, x, x[:, :1], x[:, :, :4]), lambda: api.gated_scan_bwd(x, x, x[:, :1], x.bfloat16()),
            lambda: api.gated_scan_step(x, x, state), lambda: api.gated_scan_step(x[:, 0], x[:, 0], state[:1]),
            lambda: api.gated_scan_step(x[:, 0], x[:, 0], state.double()), lambda: api.gated_scan_step(x[:, 0], x[:, 0], state[:, :4]),
            lambda: api.gated_scan_step(x[:, 0], x[:, 0], torch.zeros(8, 3).T), lambda: api.gated_scan_step(x[:, 0], x[:, 0], state, slots.long()),
            lambda: api.gated_scan_step(x[:, 0], x[:, 0], state, slots[:1]), lambda: api.gated_scan_step(x[:, 0], x[:, 0, :4], state),
            lambda: api.gated_scan_step(x[:, 0], x[:, 0], state, torch.zeros(4, dtype=torch.int32)[::2]),
            lambda: api.gated_scan_step(x[:, 0].half(), x[:, 0].half(), state),
            lambda: api.qk_norm_fwd(q[..., :12], q[..., :12]), lambda: api.qk_norm_fwd(q, q[:, :3]), lambda: api.qk_norm_fwd(q, q[:1]),
            lambda: api.qk_norm_fwd(q, one), lambda: api.qk_norm_fwd(q, q[..., :8]), lambda: api.qk_norm_fwd(q.bfloat16(), q),
            lambda: api.qk_norm_fwd(q.half(), q.half()), lambda: api.qk_norm_fwd(q.transpose(2, 3), q.transpose(2, 3)),
            lambda: api.qk_norm_fwd(q, q, w[:8]), lambda: api.qk_norm_fwd(q, q, None, w.bfloat16()),
            lambda: api.qk_norm_fwd(q, q, torch.zeros(32)[::2]), lambda: api.qk_norm_fwd(q, q, table=torch.zeros(9, 24)),
            lambda: api.qk_norm_fwd(q, q, table=torch.zeros(9, 12)), lambda: api.qk_norm_fwd(q, q, table=table[:3]),
            lambda: api.qk_norm_fwd(q, q, table=table.double()), lambda: api.qk_norm_fwd(q, q, table=torch.zeros(16, 9).T),
            lambda: api.qk_norm_fwd(one, one, table=table[:0]), lambda: api.qk_norm_fwd(q, q, positions=at),
            lambda: api.qk_norm_fwd(q, q, table=table, positions=at.long()), lambda: api.qk_norm_fwd(q, q, table=table, positions=at[0]),
            lambda: api.qk_norm_bwd(q, q, None, None, q[:, :2], q), lambda: api.qk_norm_bwd(q, q, None, None, q, q.bfloat16()),
            lambda: api.qk_norm_bwd(q, q, None, None, q, q.transpose(2, 3)))):
        with pytest.raises(ValueError):
            fn()
            raise AssertionError(f"call {i} went through")
