"""GPU tests of the gated recurrence against 64-bit formulas where a bound of the
channel's largest value would see nothing: what stands behind a new start, element by
element; what the formula leaves infinite or NaN; a long chain of tiles in full.

Tolerances as in test_gpu_lm_more.py: 400 u (u = 2^-24) of what a step's own states
and gradients are, beside one rounding to the output's type.
"""
import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300.build import build

from . import _lm_more as m
from .test_gpu_lm_more import BF16, F32, U, _gated_check, _gated_run, _views

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    build()
    b.lib()
    yield
    b.mgs_check()


# (a tile in part, a cluster over time, enough lanes for none)
@pytest.mark.parametrize("B,T,D", [(2, 60, 64), (1, 700, 66), (80, 200, 64)])
@pytest.mark.parametrize("start", [torch.inf, 30.0])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e8])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_new_start_behind_a_large_state(dtype, size, start, B, T, D):
    # the first state is large and stays, masked, up to a gate of +inf (or 30: a = 1e-13), at another step of each
    # channel: what follows knows nothing of it, and errs by its own states and gradients alone
    d = m.gated_inputs(B, T, D, dtype, positive=False, seed=T + D, shift=0.5, halves=False)
    d["h0"] = d["h0"].sign() * size
    at, step = T // 3 + torch.arange(D) % 11, torch.arange(T)[:, None]
    d["gate"] = torch.where(step < at, -torch.inf, torch.where(step == at, start, d["gate"].float())).to(dtype)
    got, ref = _gated_run(_views(d)), m.gated_ref(d)
    behind = (step > at).expand(B, T, D)
    k, before = d["gate"].double(), torch.cat([d["h0"].double()[:, None], ref["h"][:, :-1]], 1)
    away = d["value"].double().abs() + before.abs()  # what c - h comes from

    def largest(x, where):  # in each channel
        return (x.abs() * where).amax(1, keepdim=True)

    since = behind | (step == at)
    lam = largest(ref["lam"], since)
    m.check_each("h", got["h"], ref["h"], 400 * U * torch.where(since, largest(ref["h"], since), ref["h"].abs()))
    m.check_each("dvalue", got["dvalue"], ref["dvalue"], 400 * U * lam * since)
    slope = torch.sigmoid(k) * torch.sigmoid(-k)  # (0 up to the new start, 1e-13 at one of 30)
    m.check_each("dgate", got["dgate"], ref["dgate"], 400 * U * lam * torch.where(behind, largest(away, behind), away * slope))


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,D", [(2, 300, 32), (1, 2300, 34), (90, 90, 7)])
@pytest.mark.parametrize("what,x", [("value", torch.inf), ("value", -torch.inf), ("value", torch.nan), ("gate", torch.nan),
                                    ("grad_h", torch.nan), ("grad_h", torch.inf), ("h0", torch.inf), ("h0", torch.nan)])
def test_what_the_formula_leaves_infinite_or_nan(what, x, B, T, D, dtype, positive):
    # is infinite or NaN (an infinity may have become NaN), the rest is finite
    d = m.gated_inputs(B, T, D, dtype, positive=positive, seed=12, halves=False)
    d[what][(0, D // 2) if what == "h0" else (0, T * 2 // 3, D // 2)] = x
    got, ref = _gated_run(_views(d)), m.gated_ref(d)
    for n in ("h", "h_T", "dgate", "dvalue", "dh0"):
        assert torch.equal(torch.isfinite(got[n]).cpu(), torch.isfinite(ref[n])), n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_long_chain_of_tiles_in_full(dtype):
    # all states and gradients of 1563 tiles, and what the whole chain of rounds ends in
    d = m.gated_inputs(1, 100001, 2, dtype, seed=64, shift=1.0)
    _gated_check(_gated_run(_views(d)), m.gated_ref(d))


def _exchange(block, at, ns):
    rounds, wrong = (torch.full((b.EXCHANGE_BLOCKS,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    b.mgs_debug_exchange(block, at, ns, rounds, wrong)
    return rounds, wrong


def test_exchange_of_a_cluster():
    # a block that comes late, within the limit of the others' waits
    for block, at in ((-1, 0), (0, 0), (3, 2), (7, b.EXCHANGE_ROUNDS - 1)):
        rounds, wrong = _exchange(block, at, 2_000_000)
        b.mgs_check()
        assert (rounds == b.EXCHANGE_ROUNDS).all() and not wrong.any()


@pytest.mark.parametrize("block", [0, 5])
@pytest.mark.parametrize("at", range(b.EXCHANGE_ROUNDS))
def test_exchange_whose_waits_give_up(at, block):
    # past the limit: the others have pushed in that round and take no further part; the late one has their messages of
    # it and pushes once more.  Nothing is on its way when they leave, and the next call knows nothing of it.
    d = _views(m.gated_inputs(1, 1000, 64, BF16, seed=7))
    want = _gated_run(d)
    b.mgs_check()
    b.mgs_set_wait_timeout_ns(2_000_000)
    try:
        rounds, wrong = _exchange(block, at, 50_000_000)
        with pytest.raises(b.MGSError) as e:
            b.mgs_check()
        assert e.value.status == b.MGS_ERR_TIMEOUT
        b.mgs_check()  # cleared
    finally:
        b.mgs_set_wait_timeout_ns(1_000_000_000)
    took = [at + 1] * b.EXCHANGE_BLOCKS
    took[block] = min(at + 2, b.EXCHANGE_ROUNDS)
    assert rounds.tolist() == took and not wrong.any()
    for n, x in _gated_run(d).items():
        assert torch.equal(x, want[n]), n
