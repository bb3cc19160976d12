"""The projections in few bits have no gradients: inputs that ask for one are
refused, not answered with results cut off from them (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")


def calls():
    from selective_state_space_63_amd import q4
    x, w, s = torch.zeros(3, 128), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    xs, nw, r, gamma = torch.ones(3), torch.ones(128), torch.zeros(3, 128), torch.ones(128)
    linear = lambda **k: q4.q4_linear(**{**dict(x=x, weight=w, scales=s), **k})  # noqa: E731
    norm = lambda **k: q4.add_norm_q8_fwd(**{**dict(x=x, weight=nw, residual=r, gamma=gamma), **k})  # noqa: E731
    return [(linear, "x", x), (linear, "scales", s), (linear, "x_scale", xs), (norm, "x", x), (norm, "weight", nw),
            (norm, "residual", r), (norm, "gamma", gamma)]


@pytest.mark.parametrize("which", range(7))
def test_inputs_that_require_a_gradient_are_refused(which):
    call, name, value = calls()[which]
    leaf = value.clone().requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        call(**{name: leaf})
    # otherwise the checks go on to the next thing that is wrong here: no device
    for ask in (lambda: call(**{name: leaf.detach()}), lambda: torch.no_grad()(call)(**{name: leaf}),
                lambda: torch.inference_mode()(call)(**{name: leaf})):
        with pytest.raises(ValueError, match="device|8-bit"):
            ask()
