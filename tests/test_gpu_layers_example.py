"""The example with the gated recurrence among its layers and with 4-bit
weights: the operators together, as they are used.

Bars.  A prompt followed by single tokens against the whole sequence: as in the
example's first test, 24 * 2^-9 (bf16) and 24 * 2^-16 (fp32) of the logits' norm.
4-bit weights against the same model with the weights that the codes stand for
in place of its own: the two differ by the rounding of the norms' outputs to 8
bits, which is off by half a step, 2^-4 of a value at most and 2^-4 / sqrt(3) of
the norm as a whole (errors spread evenly over the step), once in each of two layers;
what a layer makes of it (gates, decays, products of two projections) passes it
on up to four times (two factors in which it is linear, each with the same
error): 2 * 4 * 2^-4 / sqrt(3) = 0.29.
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


def off(got, want):
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kinds", [("gated",), ("heads", "gated")], ids="-".join)
def test_trains_and_decodes(example, dtype, kinds):
    import torch
    torch.manual_seed(2)
    model = example.Model(dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, kinds=kinds).cuda()
    before = {n: p.detach().clone() for n, p in model.named_parameters()}
    losses = example.train(model, 5)
    assert all(math.isfinite(v) for v in losses)
    for n, p in model.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()) and float(p.grad.abs().max()) > 0, n
        assert not torch.equal(before[n], p), n
    tokens = torch.randint(32, (3, 200), device="cuda")
    for prompt in (1, 64, 128, 199):
        got = example.prompt_then_tokens(model, tokens, prompt)
        with torch.no_grad():
            want = model(tokens)[0][:, prompt:]
        assert off(got, want) <= (24 * 2.0 ** -9 if dtype == "bf16" else 24 * 2.0 ** -16), prompt


def test_gradients_against_differences(example):
    """The loss along a direction of all parameters (fp32 layers).  Central
    differences over 2 e of an fp32 loss of about 4: its roundings, 2^-22, over
    2 e = 4e-3 make 6e-5, the third order some e^2; the gradient's own error is
    the fp32 bar of the sums, far below.  Allowed: 1e-3 of the larger of the
    gradient's length and 1."""
    import torch
    from torch.nn import functional as F
    torch.manual_seed(3)
    model = example.Model(dtype=torch.float32, kinds=("heads", "gated")).cuda()
    tokens = torch.randint(32, (4, 150), device="cuda")

    def loss():
        return F.cross_entropy(model(tokens)[0][:, 2:].flatten(0, 1).double(), tokens[:, :-2].flatten())

    loss().backward()
    params = list(model.parameters())
    length = math.sqrt(sum(float(p.grad.double().square().sum()) for p in params))
    # along the gradient itself, where the change is largest
    e = 2e-3
    values = []
    with torch.no_grad():
        for s in (e, -e):
            for p in params:
                p.add_(p.grad, alpha=s / length)
            values.append(float(loss()))
            for p in params:
                p.add_(p.grad, alpha=-s / length)
    assert abs((values[0] - values[1]) / (2 * e) - length) <= 1e-3 * max(length, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_four_bit_weights(example, dtype):
    import torch
    torch.manual_seed(4)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    model = example.Model(dtype=dt, kinds=("heads", "gated")).cuda()
    tokens = torch.randint(32, (40, 60), device="cuda")  # 40 sequences: more rows than the first product kernel takes
    for layer in model.layers:
        layer.pack()
    got = {n: example.prompt_then_tokens(model, tokens[:n], 40) for n in (1, 3, 40)}
    assert torch.equal(got[3], example.prompt_then_tokens(model, tokens[:3], 40))
    # the model with the weights that the codes stand for, in its own type
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    values = torch.cat([values, -values])
    with torch.no_grad():
        whole = [model(tokens[:n, :40])[1] for n in (1, 3, 40)]   # states of the prompts, before the weights change
        for layer in model.layers:
            for name, (code, scale) in zip(("w_in", "w_out"), layer.packed):
                w = values[torch.stack([code & 15, code >> 4], -1).flatten(-2).long()]
                w = (w.unflatten(-1, (scale.shape[1], -1)) * scale.float()[..., None]).flatten(-2)
                getattr(layer, name).copy_(w)
            layer.packed = None
        for n, states in zip((1, 3, 40), whole):
            want = torch.stack([model.step(tokens[:n, t], states) for t in range(40, 60)], 1)
            assert off(got[n], want) <= 0.29, (n, off(got[n], want))
