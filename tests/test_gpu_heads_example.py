"""The example that runs the block operators together: it trains, and a prompt
followed by single tokens gives the logits of the whole sequence.

Bars: each of the two ways rounds about eight values per layer (the input
projection's row, the scan's y, the norms' outputs, the output projection) to
the dtype, independently and to 2^-9 (bf16) each; two layers, both ways and
the head's own projection make about 36 such roundings, which add as their root:
6 * 2^-9, taken with a factor of 4.  fp32: the scans' bar, 2^-16, taken with
the same factor of 24.
"""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("heads_block",
                                                  os.path.join(HERE, "..", "examples", "heads_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_trains_and_decodes(example, dtype):
    import torch
    torch.manual_seed(1)
    model = example.Model(dtype=torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    losses = example.train(model, 60)
    assert all(math.isfinite(v) for v in losses)
    assert sum(losses[-5:]) < 0.9 * sum(losses[:5])
    for n, p in model.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()) and float(p.grad.abs().max()) > 0, n
    tokens = torch.randint(32, (3, 90), device="cuda")
    for prompt in (1, 64, 89):
        got = example.prompt_then_tokens(model, tokens, prompt)
        with torch.no_grad():
            want = model(tokens)[0][:, prompt:]
        err = float((got - want).norm() / want.norm())
        assert err <= (24 * 2.0 ** -9 if dtype == "bf16" else 24 * 2.0 ** -16), (prompt, err)
