"""The workspace of every scan belongs to the stream that the call names: one of
torch's current stream would be handed out again while the kernels still use it.
Without a GPU: the library's entry points are replaced."""
import contextlib

import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300 import api

Z = torch.zeros
MAT, VEC, INIT = Z(2, 3, 1, 8, 8), Z(2, 3, 1, 8), Z(2, 1, 8)
ANG, LANES, QKV = Z(2, 3, 1, 28), Z(2, 3, 4), Z(2, 3, 1, 64)
CALLS = {
    "mgs_matrix_affine_scan_fwd": lambda s: api.matrix_affine_scan_fwd(MAT, VEC, INIT, stream=s),
    "mgs_matrix_affine_scan_bwd": lambda s: api.matrix_affine_scan_bwd(MAT, INIT, VEC, VEC, stream=s),
    "mgs_matrix_affine_scan_bwd_recompute": lambda s: api.matrix_affine_scan_bwd_recompute(MAT, VEC, INIT, VEC, stream=s),
    "mgs_matrix_scan_fwd": lambda s: api.matrix_scan_fwd(MAT, stream=s),
    "mgs_matrix_scan_bwd": lambda s: api.matrix_scan_bwd(MAT, MAT, MAT, stream=s),
    "mgs_parallel_scan_log_bwd": lambda s: api.parallel_scan_log_bwd(LANES, LANES, None, None, LANES, stream=s),
    "mgs_givens_affine_scan_fwd": lambda s: api.givens_affine_scan_fwd(ANG, VEC, VEC, stream=s),
    "mgs_givens_affine_scan_bwd": lambda s: api.givens_affine_scan_bwd(ANG, VEC, None, VEC, VEC, stream=s),
    "mgs_givens_matrix_scan_fwd": lambda s: api.givens_matrix_scan_fwd(ANG, stream=s),
    "mgs_givens_matrix_scan_bwd": lambda s: api.givens_matrix_scan_bwd(ANG, MAT, MAT, stream=s),
    "mgs_delta_scan_fwd": lambda s: api.delta_scan_fwd(QKV, QKV, QKV, Z(2, 3, 1), stream=s),
    "mgs_linear_scan_fwd": lambda s: api.linear_scan_fwd(LANES, LANES, stream=s),
    "mgs_linear_scan_bwd": lambda s: api.linear_scan_bwd(LANES, None, LANES, LANES, stream=s),
}


@pytest.mark.parametrize("stream,name", [("side", "side"), (7, ("external", 7)), (0, "default"), (None, "current")])
@pytest.mark.parametrize("entry", CALLS)
def test_workspace_belongs_to_the_named_stream(monkeypatch, entry, stream, name):
    current, taken, calls = ["current"], [], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    empty = torch.empty

    def new(*a, **k):
        if k.get("dtype") is torch.uint8:
            taken.append(current[-1])
        return empty(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda at, device=None: ("external", at))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", new)
    monkeypatch.setattr(api, "_check", lambda *a, **k: None)
    monkeypatch.setattr(b, "mgs_workspace_size", lambda *a: 256)
    monkeypatch.setattr(b, entry, lambda *a: calls.append(a))
    CALLS[entry](stream)
    assert taken == [name] and len(calls) == 1 and calls[0][-1] is stream
