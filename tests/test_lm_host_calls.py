"""What the tensor-level functions of the language-model operators do around a
call of the library, without a GPU: the library's entry points are replaced."""
import contextlib

import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api

from . import _lm

BF16 = torch.bfloat16


class _Calls:
    """The entry points' calls, and the streams that were torch's current ones when memory was taken or copied."""

    def __init__(self, monkeypatch):
        self.current, self.copies, self.scratch, self.calls = ["current"], [], [], []

        @contextlib.contextmanager
        def on(stream):
            self.current.append(stream)
            yield
            self.current.pop()

        dense, empty = torch.Tensor.contiguous, torch.empty

        def contiguous(t):
            if not t.is_contiguous():
                self.copies.append(self.current[-1])
            return dense(t)

        def new(*a, **k):
            if k.get("dtype") is torch.uint8:
                self.scratch.append(self.current[-1])
            return empty(*a, **k)

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, device=None: ("external", at))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
        monkeypatch.setattr(torch.Tensor, "contiguous", contiguous)
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
        monkeypatch.setattr(torch, "empty", new)
        monkeypatch.setattr(api, "_check_typed", lambda *a, **k: None)
        monkeypatch.setattr(b, "mgs_linear_attention_workspace_size", lambda shape, backward: 256)
        for name in ("mgs_linear_attention_fwd", "mgs_linear_attention_bwd"):
            monkeypatch.setattr(b, name, lambda *a, _name=name: self.calls.append((_name, a)))


@pytest.mark.parametrize("stream,name", [(1234, ("external", 1234)), (0, "default"), ("a torch stream", "a torch stream"),
                                         (None, "current")])
def test_copies_and_workspace_belong_to_the_named_stream(monkeypatch, stream, name):
    # a copy on another stream than the kernels' could be read before it is written, and its memory or the
    # workspace's be handed out again while they run
    d = _lm.attn_inputs(2, 8, 2, 2, 64, BF16, S0=False)
    calls = _Calls(monkeypatch)
    q = d["q"][:, :1].expand(2, 8, 2, 64)
    go = d["grad_o"][:1, :1].expand(2, 8, 2, 64)
    api.linear_attention_fwd(q, d["k"], d["v"], d["g"], stream=stream)
    api.linear_attention_bwd(d["q"], d["k"], d["v"], d["g"], go, stream=stream)
    assert [n for n, _ in calls.calls] == ["mgs_linear_attention_fwd", "mgs_linear_attention_bwd"]
    assert calls.copies == [name, name] and calls.scratch == [name, name]
    assert all(a[-1] is stream for _, a in calls.calls)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_broadcast_queries_and_keys_are_copied_where_it_matters(monkeypatch, dtype):
    # no tensor map has a zero stride: the library would take its slow kernel (fp32's forward reads q, k and v
    # through tensors of its own)
    d = _lm.attn_inputs(2, 8, 2, 2, 64, dtype, S0=False)
    calls = _Calls(monkeypatch)
    q, k = (d[n][:, :1].expand(2, 8, 2, 64) for n in ("q", "k"))
    api.linear_attention_fwd(q, k, d["v"], d["g"])
    api.linear_attention_bwd(q, k, d["v"], d["g"], d["grad_o"])
    (_, fwd), (_, bwd) = calls.calls
    assert all(0 not in t.stride() for t in bwd[1:3])
    assert all((0 not in t.stride()) == (dtype == BF16) for t in fwd[1:3])


def test_tensors_written_in_place_are_marked_for_autograd(monkeypatch):
    d = _lm.attn_inputs(2, 1, 2, 2, 64, BF16)
    _Calls(monkeypatch)
    monkeypatch.setattr(b, "mgs_linear_attention_step", lambda *a: None)
    q, k, v, g = (d[n][:, 0] for n in ("q", "k", "v", "g"))
    S, out = d["S0"], torch.zeros(2, 2, 64, dtype=BF16)
    before = [t._version for t in (S, out, q)]
    api.linear_attention_step(q, k, v, g, S, out=out)
    assert [t._version for t in (S, out, q)] == [before[0] + 1, before[1] + 1, before[2]]
    with torch.inference_mode():
        cache = torch.zeros(2, 2, 64, 64)
    api.linear_attention_step(q, k, v, g, cache)  # an inference tensor has no version
    # what is differentiated keeps its state: a step on it is noticed
    S = torch.ones(3, requires_grad=True) * 2
    loss = (S * S).sum()
    api._written([S])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_clipped_tensors_are_marked_for_autograd(monkeypatch):
    monkeypatch.setattr(b, "mgs_clip_grad_norm_workspace_size", lambda n: 0)
    monkeypatch.setattr(b, "mgs_clip_grad_norm", lambda *a: None)
    grads, outs = [torch.zeros(8), torch.zeros(3, dtype=BF16)], [torch.zeros(8), torch.zeros(3, dtype=BF16)]

    class Card:  # the first check asks for the device's type alone
        type = "cuda"
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: Card()))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    api.clip_grad_norm(grads, 1.0, out=outs)
    assert [t._version for t in grads + outs] == [0, 0, 1, 1]
    api.clip_grad_norm(grads, 1.0)
    assert [t._version for t in grads + outs] == [1, 1, 1, 1]


def test_second_derivatives_are_refused(monkeypatch):
    # the gradients come out of the library without a graph of their own: a second differentiation would take
    # them for constants
    monkeypatch.setattr(api, "linear_attention_fwd", lambda q, k, v, g, S0, scale, want_state: (v.detach() * 2, v.detach().sum()))
    monkeypatch.setattr(api, "linear_attention_bwd", lambda q, k, v, g, go, S0, gST, scale: (q * 0, k * 0, go.detach() * 2, None, None))
    monkeypatch.setattr(api, "rms_norm_fwd", lambda x, w, res, eps: (x.detach() * 2, x.detach(), x.detach()))
    monkeypatch.setattr(api, "rms_norm_bwd", lambda r, w, rstd, gy, gr: (gy.detach() * r, w * 0))
    q, w = torch.ones(1, 2, 1, 64, requires_grad=True), torch.ones(64, requires_grad=True)
    for y in (api.linear_attention(q, q, q, torch.zeros(1, 2, 1))[0], api.rms_norm(q, w)):
        d, = torch.autograd.grad((y * y).sum(), q, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            ((d * d).sum() + (q * q).sum()).backward()
