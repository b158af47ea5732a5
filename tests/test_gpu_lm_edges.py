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
