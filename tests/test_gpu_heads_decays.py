"""The multi-head scan and its gradients where the decays are strong: resets of
packed sequences, several in a chunk, heads that forget within a token, and
decays of infinite strength.

The bars are those of test_gpu_heads_scan.py, as multiples of each value's
magnitude (the sum of its terms' absolute values, decayed as the terms are).
They hold here because a decay between two tokens is exact to 2^-24 times the
exponents between those two, whatever the chunk holds beside them: a value with
a magnitude above 1e-30 has exponents below 100 (in units of ln 2), formed with
three roundings, 100 * 3 * 2^-24 * ln 2 = 0.8 * 2^-16.
"""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_heads_scan import F32_BAR, bar, case, close, fwd, opts, torch_cuda  # noqa: F401

pytestmark = pytest.mark.gpu


def both(torch, d, n, step, unit, dtype, seed, want=None, dh=True):
    """Forward and gradients against the reference of `want` (the inputs in 64
    bits, n unless given)."""
    from selective_state_space_63_amd import block
    want = n if want is None else want
    y, hl = fwd(d, step, unit)
    ry, my, rh, mh = ref.scan(want["x"], want["delta"], want["A"], want["Bm"], want["Cm"], want["D"], want["h0"],
                              want["bias"], step == "softplus", unit)
    close(y, ry, my, bar(dtype), "y")
    close(hl, rh, mh, bar(dtype, True), "h_last")
    g = np.random.default_rng(seed)
    dy = torch.from_numpy(g.standard_normal(tuple(d["x"].shape)).astype(np.float32)).cuda().to(d["x"].dtype)
    dl = torch.from_numpy(g.standard_normal(rh.shape).astype(np.float32)).cuda() if dh else None
    got = block.heads_scan_bwd(d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], dy, dh_last=dl, **opts(d, step, unit))
    torch.cuda.synchronize()
    rb = ref.scan_bwd(want["x"], want["delta"], want["A"], want["Bm"], want["Cm"], dy.double().cpu().numpy(), want["D"],
                      want["h0"], None if dl is None else dl.double().cpu().numpy(), want["bias"], step == "softplus",
                      unit)
    for k in sorted(got):
        close(got[k], *rb[k], bar(dtype, k not in ("dx", "dBm", "dCm", "ddelta")), k)


def resets(d, n, where, value=3.0e3):
    """Steps that start a sequence anew, in both copies of the inputs."""
    for t in where:
        d["delta"][:, t] = value
        n["delta"][:, t] = float(d["delta"][0, t, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_with_many_resets(torch_cuda, dtype):
    """Short sequences packed one after another, up to twenty in 64 tokens: each
    is what it is alone."""
    torch = torch_cuda
    d, n = case(torch, 2, 200, 2, 64, 1, 64, dtype, "delta", True, 31)
    at = sorted(set(range(1, 64, 3)) | {70, 75, 76, 77, 100, 127, 128, 129, 150, 191, 192})
    resets(d, n, at)
    y, hl = fwd(d, "delta", True)
    ry, my, rh, mh = ref.scan(n["x"], n["delta"], n["A"], n["Bm"], n["Cm"], n["D"], n["h0"], None, False, True)
    close(y, ry, my, bar(dtype), "y")
    close(hl, rh, mh, bar(dtype, True), "h_last")
    ends = at + [200]
    for lo, hi in zip(at, ends[1:]):
        part = {k: (v[:, lo:hi] if k in ("x", "Bm", "Cm", "delta") else v) for k, v in n.items()}
        ry, my, _, _ = ref.scan(part["x"], part["delta"], part["A"], part["Bm"], part["Cm"], part["D"], None, None, False,
                                True)
        close(y[:, lo:hi], ry, my, bar(dtype), f"y from {lo}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("unit", [True, False])
@pytest.mark.parametrize("a", [-4.0, -8.0, -12.0, -16.0, -20.0])
def test_strong_decays(torch_cuda, dtype, unit, a):
    """Heads that forget within a token beside one that does not."""
    torch = torch_cuda
    d, n = case(torch, 1, 150, 3, 24, 1, 32, dtype, "softplus", True, 32)
    d["bias"].fill_(0.6)   # steps of about 1
    n["bias"][:] = np.float32(0.6)
    A = np.array([a, 0.75 * a, -1e-3], np.float32)
    d["A"].copy_(torch.from_numpy(A))
    n["A"] = A.astype(np.float64)
    both(torch, d, n, "softplus", unit, dtype, 33)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [3.0e3, 1.0e30])
def test_gradients_with_resets(torch_cuda, dtype, value):
    """Sequences packed one after another: nothing reaches across a reset, and
    the reset's own step has no gradient."""
    torch = torch_cuda
    d, n = case(torch, 2, 300, 2, 64, 1, 64, dtype, "delta", True, 34)
    resets(d, n, (0, 1, 17, 40, 63, 64, 130, 131, 160, 255, 256, 299), value)
    both(torch, d, n, "delta", True, dtype, 35)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_with_infinite_steps(torch_cuda, dtype):
    """A reset by a step of +infinity: the limit of large steps, whose gradients
    are 0 at that token and what they are without it elsewhere."""
    torch = torch_cuda
    d, n = case(torch, 1, 150, 2, 64, 1, 64, dtype, "delta", True, 36)
    for t in (50, 97, 128):
        d["delta"][:, t] = float("inf")
        n["delta"][:, t] = 1.0e30
    both(torch, d, n, "delta", True, dtype, 37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("unit", [True, False])
def test_gradients_with_infinite_decay(torch_cuda, dtype, unit):
    """A head with A = -infinity keeps nothing: its decay has no gradient."""
    torch = torch_cuda
    d, n = case(torch, 2, 140, 2, 16, 1, 16, dtype, "softplus", True, 38)
    d["A"][1] = float("-inf")
    n["A"][1] = -1.0e30
    both(torch, d, n, "softplus", unit, dtype, 39)
