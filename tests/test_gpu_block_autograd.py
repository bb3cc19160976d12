"""What torch autograd is told about the operators: that their gradients have
none of their own, which gradients are asked for, and what is written in place."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_63_amd import s6
    s6.load_library()
    return torch


def heads_inputs(torch, dtype=None):
    g = torch.Generator("cuda").manual_seed(71)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return dict(x=r(2, 40, 4, 16), delta=0.1 * r(2, 40, 4).abs(), A=-torch.rand(4, device="cuda") - 0.1,
                Bm=r(2, 40, 1, 16), Cm=r(2, 40, 1, 16), D=r(4), h0=r(2, 4, 16, 16), bias=0.1 * r(4).abs())


def test_gradients_of_gradients_are_refused(torch_cuda):
    """A penalty on a gradient needs second derivatives, which there are not: an
    error, not a constant."""
    from selective_state_space_63_amd import block, s6
    torch = torch_cuda
    d = heads_inputs(torch)
    leaf = lambda t: t.clone().requires_grad_()  # noqa: E731
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    calls = []
    x = leaf(d["x"])
    calls.append((block.HeadsScan.apply(x, d["delta"], d["A"], d["Bm"], d["Cm"])[0], x))
    v = leaf(r(6, 32))
    calls.append((block.AddNorm.apply(v, torch.ones(32, device="cuda"))[0], v))
    u = leaf(r(6, 32))
    calls.append((block.GatedNorm.apply(u, r(6, 32), torch.ones(32, device="cuda")), u))
    z = leaf(r(2, 32, 24))
    calls.append((s6.SelectiveScan.apply(z, r(2, 32, 24).abs(), -r(32, 8).abs(), r(2, 8, 24), r(2, 8, 24)), z))
    for out, inp in calls:
        g, = torch.autograd.grad((out * out).sum(), inp, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable|twice"):
            (g * g).sum().backward()
