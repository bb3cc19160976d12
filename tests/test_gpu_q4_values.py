"""Products with 4-bit weights (include/s6_q4.h) of values at the ends of their
types: what a group's scale makes small stays finite before it does."""
import math

import numpy as np
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


@pytest.mark.parametrize("m", [1, 6, 16, 40, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_rows_and_small_scales(torch_cuda, dtype, group, m):
    """Rows near the largest number, the largest value of a code, scales that bring
    the result back.  Bar: 2^-24 (16 + sqrt(K)) of the sum of the terms' absolute
    values, a rounding of the result's type besides."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    print(f"[case] q4 large rows {m} {group} {dtype}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, n = 256, 48
    g = np.random.default_rng([91, m, group])
    x = torch.from_numpy((g.uniform(1e38, 3.3e38, (m, k)) * g.choice([-1, 1], (m, k))).astype(np.float32)).cuda().to(dt)
    x[0] = x[0].abs()                                   # one row whose terms all add up
    w = torch.full((n, k // 2), 0x77, dtype=torch.uint8, device="cuda")          # 6 everywhere
    w[1] = 0x7f                                                                  # -6 and 6 in turn
    s = torch.from_numpy(g.uniform(1e-6, 1e-4, (n, k // group)).astype(np.float32)).cuda().to(torch.bfloat16)
    y = q4.q4_linear(x, w, s, out_dtype=torch.float32)
    v = np.full((n, k), 6.0)
    v[1, 0::2] = -6.0
    W = v * np.repeat(s.double().cpu().numpy(), group, 1)
    X = x.double().cpu().numpy()
    want, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    got = y.double().cpu().numpy()
    assert mag.max() < 2.0 ** 127 and np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -24 * (16 + math.sqrt(k)) * mag + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_rows_and_large_scales(torch_cuda, dtype, group, m):
    """Rows of the smallest numbers, scales that bring the result back.  The third
    bf16 part of an fp32 x rounds to a multiple of 2^-133: 2^-134 of each x is
    allowed besides; products are exact."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    print(f"[case] q4 small rows {m} {group} {dtype}", flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, n = 256, 48
    g = np.random.default_rng([92, m, group])
    x = torch.from_numpy((g.standard_normal((m, k)) * 2.0 ** g.uniform(-125, -90, (m, 1))).astype(np.float32)).cuda().to(dt)
    codes = g.integers(0, 256, (n, k // 2), dtype=np.uint8)
    s = torch.from_numpy((2.0 ** 100 * g.uniform(0.5, 1, (n, k // group))).astype(np.float32)).cuda().to(torch.bfloat16)
    y = q4.q4_linear(x, torch.from_numpy(codes).cuda(), s, out_dtype=torch.float32)
    values = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
    v = values[np.stack([codes & 15, codes >> 4], -1).reshape(n, k)]
    S = np.repeat(s.double().cpu().numpy(), group, 1)
    X = x.double().cpu().numpy()
    want, mag = X @ (v * S).T, np.abs(X) @ np.abs(v * S).T
    lost = (2.0 ** -134 if dtype == "f32" else 0.0) * np.abs(v * S).sum(1)
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -24 * (16 + math.sqrt(k)) * mag + 2.0 ** -24 * np.abs(want) + lost).all()
