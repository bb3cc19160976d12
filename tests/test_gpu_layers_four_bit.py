"""The example's single tokens with 4-bit weights against the same layers with
the products formed in 64 bits from the same codes, scales and 8-bit rows: what
is left is the sums' order and one rounding of a product's result.

Bar: as prompts against single tokens in the example's tests, 24 * 2^-9 (bf16) and
24 * 2^-16 (fp32) of the logits' norm."""
import pytest

from test_gpu_layers_example import example, off  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 3, 40])
@pytest.mark.parametrize("kinds", [("gated",), ("heads", "gated")], ids="-".join)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products_of_the_layers(example, monkeypatch, dtype, kinds, batch):  # noqa: F811
    import torch
    print(f"[case] four-bit layers {dtype} {kinds} {batch}", flush=True)
    torch.manual_seed(5)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    model = example.Model(dtype=dt, kinds=kinds).cuda()
    tokens = torch.randint(32, (batch, 50), device="cuda")
    for layer in model.layers:
        layer.pack()
    got = example.prompt_then_tokens(model, tokens, 40)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float64)
    values = torch.cat([values, -values])
    calls = []

    def plain(x, weight, scales, x_scale=None, out_dtype=None, y=None):
        calls.append(x.dtype)
        w = values[torch.stack([weight & 15, weight >> 4], -1).flatten(-2).long()]
        w = (w.unflatten(-1, (scales.shape[1], -1)) * scales.double()[..., None]).flatten(-2)
        out = torch.matmul(x.double(), w.t().contiguous())
        if x_scale is not None:
            out = out * x_scale.double()[..., None]
        return out.to(out_dtype or x.dtype)

    monkeypatch.setattr(example.q4, "q4_linear", plain)
    want = example.prompt_then_tokens(model, tokens, 40)
    assert len(calls) == 10 * 2 * len(model.layers) and torch.float8_e4m3fn in calls
    assert off(got, want) <= (24 * 2.0 ** -9 if dtype == "bf16" else 24 * 2.0 ** -16), off(got, want)
