"""The example that trains and serves a small model on the language-model operators."""
import pytest
import torch

from scan_linear_recurrences_gb300 import _binding as b
from scan_linear_recurrences_gb300.build import build

pytestmark = pytest.mark.gpu


def test_example_learns_and_serves():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    build()
    from examples import linear_attention_lm as ex
    torch.manual_seed(0)
    model = ex.Model().to("cuda", torch.bfloat16)
    losses = ex.train(model, 40)
    # the last loss is below that of a model without memory (ln 64), the first is above it
    assert losses[0] > 4.1 and sum(losses[-5:]) / 5 < 3.9
    # a prompt and then single tokens give the logits of the whole as one prompt: the same formulas in other
    # orders of summation, with about ten roundings to bf16 on the way (2^-9 each) and one to 8 bits whose
    # steps (2^-4) some of the differences cross
    for layer in model.layers:
        layer.freeze()
    text, _ = ex.texts(3, 140, 64, torch.Generator().manual_seed(5))
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    whole = model.serve(text, model.cache(5), slots)
    cache = model.cache(5)
    got = [model.serve(text[:, :130], cache, slots)[:, -1]]
    for t in range(130, 140):
        got.append(model.serve(text[:, t], cache, slots))
    got, want = torch.stack(got, 1).double(), whole[:, 129:].double()
    assert ((got - want).norm() / want.norm()).item() < 0.05
    assert not cache[0][[1, 3]].any() and cache[0][slots.long()].any()
    b.mgs_check()
