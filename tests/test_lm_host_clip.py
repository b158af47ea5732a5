"""Clipping by the global norm refuses tensors that it would write over another:
fake addresses, which nothing reads."""
import random

import pytest

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300.build import build

FAKE = 1 << 40
F32, BF16 = b.MGS_F32, b.MGS_BF16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def _refused(ins, outs, sizes, types=None):
    """Whether it is for its ranges: without a workspace every call is refused, the legal ones for that."""
    with pytest.raises(b.MGSError) as e:
        b.mgs_clip_grad_norm(ins, outs, sizes, types or [F32] * len(ins), 1.0, FAKE << 1, None, 0, stream=0)
    assert e.value.status in (b.MGS_ERR_INVALID_ARG, b.MGS_ERR_WORKSPACE)
    return e.value.status == b.MGS_ERR_INVALID_ARG


def test_clip_refuses_what_it_would_write_over():
    a, c, d = FAKE, FAKE + 4096, FAKE + 8192
    assert not _refused([a, c], [a, c], [1024, 1024])            # in place, one behind the other
    assert not _refused([c, a], [c, a], [1024, 1024])
    assert _refused([a, a], [a, a], [1024, 1024])                # one tensor twice in place
    assert _refused([a, a + 4092], [a, a + 4092], [1024, 1024])
    assert _refused([a, c], [c, a], [1024, 1024])                # each into the other
    assert _refused([a, c], [d, a + 2048], [1024, 8])            # an output over the other's input
    assert _refused([a, c], [d, d], [1024, 1024])                # one output for both
    assert _refused([a, c], [d, d + 2046], [1024, 8], [BF16, BF16])
    assert not _refused([a, c], [d, d + 2048], [1024, 8], [BF16, BF16])
    assert not _refused([a, a], [c, d], [1024, 1024])            # one tensor into two
    assert not _refused([a, a + 8], [c, d], [1024, 100])         # overlapping inputs are only read
    assert _refused([a, a + 8], [c, a + 8], [1024, 1])           # ... one of them written
    assert not _refused([a, a, a], [a, a, a], [1024, 0, 0])      # empty ones lie nowhere
    assert not _refused([], [], [])


@pytest.mark.parametrize("n", [2, 7, 300])
def test_clip_finds_any_pair_that_meets(n):
    # as a comparison of all pairs finds it
    rng = random.Random(n)
    seen = set()
    for _ in range(200):
        span = 40 * n * n if rng.random() < 0.5 else 4 * n
        at = lambda: FAKE + 4 * rng.randrange(span)  # noqa: E731
        sizes = [rng.randrange(0, 4) for _ in range(n)]
        ins = [at() for _ in range(n)]
        outs = [i if rng.random() < 0.5 else at() for i in ins]
        meets = lambda x, nx, y, ny: nx and ny and x < y + 4 * ny and y < x + 4 * nx  # noqa: E731
        bad = any(meets(outs[i], sizes[i], outs[j], sizes[j]) for i in range(n) for j in range(i))
        bad = bad or any(meets(outs[i], sizes[i], ins[j], sizes[j]) for i in range(n) for j in range(n)
                         if i != j or ins[i] != outs[i])
        seen.add(bool(bad))
        assert _refused(ins, outs, sizes) == bool(bad)
    assert seen == {False, True}
