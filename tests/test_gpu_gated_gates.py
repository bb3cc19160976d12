"""The gates of the gated recurrence (include/s6_gated.h) where they are hard to
form: gates and biases that cancel, and gates far open, whose gradients have the
factor 1 - r; and values that enter no gradient.

Bars: bar(L) of gated_ref.py.  1 - r is e r with e = e^{-z}, z = g + bias: a sum
and two products that round once each, each off by |z| 2^-24 in the exponent.
bar(1) = 20 * 2^-23 covers those 1.5 |z| 2^-23 once the magnitude counts 1 + |z| / 8
times.  1 - r below 2^-126 (z above about 87) is 0 or not in fp32.
"""
import numpy as np
import pytest

import gated_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_63_amd import s6
    s6.load_library()
    return torch


def rows(torch, g, shape, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).cuda().to(dt)


@pytest.mark.parametrize("unit", [False, True], ids=["root", "unit"])
@pytest.mark.parametrize("dim,dtype", [(66, "bf16"), (33, "bf16"), (34, "f32"), (33, "f32")])
def test_gate_and_bias_cancel(torch_cuda, dim, dtype, unit):
    """A gate and a bias whose sum is exact give the bits of a gate that is the
    sum, whatever their sizes."""
    from selective_state_space_63_amd import gated
    torch = torch_cuda
    print(f"[case] gate and bias cancel {dim} {dtype} {unit}", flush=True)
    b, L = 2, 150
    g = np.random.default_rng([71, dim])
    x, dy = rows(torch, g, (b, L, dim), dtype), rows(torch, g, (b, L, dim), dtype)
    A = -torch.from_numpy(g.uniform(0.05, 0.5, dim).astype(np.float32)).cuda()
    # multiples of 4 up to 12 beside 1000: exact in bf16, alone and in sum
    near = [torch.from_numpy(4.0 * g.integers(-2, 3, (b, L, dim))).cuda().to(x.dtype) for _ in range(2)]
    far = [(v.float() + s).to(x.dtype) for v, s in zip(near, (1000, -1000))]
    bias = [torch.full((dim,), s, device="cuda") for s in (-1000.0, 1000.0)]
    for n, f, c in zip(near, far, bias):
        assert torch.equal(f.float() + c, n.float())
    zero = torch.zeros(dim, device="cuda")
    h0 = torch.from_numpy(g.standard_normal((b, dim)).astype(np.float32)).cuda()

    def call(gates, biases):
        k = dict(x=x, gate_a=gates[0], gate_x=gates[1], A=A, bias_a=biases[0], bias_x=biases[1], unit_input=unit)
        out = gated.gated_scan_bwd(**k, h0=h0, dy=dy)
        out["y"], out["h_last"] = gated.gated_scan_fwd(**k, h0=h0, return_last_state=True)
        h = h0.clone()
        out["token"] = gated.gated_state_update(h, x[:, 0], gates[0][:, 0], gates[1][:, 0], A, bias_a=biases[0],
                                                bias_x=biases[1], unit_input=unit)
        return dict(out, h=h)

    want, got = call(near, (zero, zero)), call(far, bias)
    for n in want:
        assert torch.equal(want[n], got[n]), n


def slopes(z):
    """sigmoid(z) and its slope r (1 - r), the latter without cancellation."""
    r = ref.sigmoid(z)
    return r, r * ref.sigmoid(-z)


@pytest.mark.parametrize("unit", [False, True], ids=["root", "unit"])
@pytest.mark.parametrize("dim,dtype", [(66, "bf16"), (33, "f32")])
@pytest.mark.parametrize("lo,hi", [(-1, 1), (4, 12), (8, 25), (25, 86), (86, 120), (-25, -4)])
def test_open_gates(torch_cuda, lo, hi, dim, dtype, unit):
    """Gradients of the gates and biases within the bar of their own size, the
    factor 1 - r in it."""
    from selective_state_space_63_amd import gated
    torch = torch_cuda
    print(f"[case] open gates {lo} {hi} {dim} {dtype} {unit}", flush=True)
    b, L = 2, 150
    g = np.random.default_rng([72, dim, lo + 200])
    x, dy = rows(torch, g, (b, L, dim), dtype), rows(torch, g, (b, L, dim), dtype)
    ga, gx = (torch.from_numpy(g.uniform(lo, hi, (b, L, dim)).astype(np.float32)).cuda().to(x.dtype) for _ in range(2))
    A = -torch.from_numpy(g.uniform(0.05, 0.5, dim).astype(np.float32)).cuda()
    ba, bx = (torch.from_numpy((0.25 * g.standard_normal(dim)).astype(np.float32)).cuda() for _ in range(2))
    got = gated.gated_scan_bwd(x, ga, gx, A, dy, bias_a=ba, bias_x=bx, unit_input=unit)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    X, GA, GX, DY, W, BA, BX = (f64(t) for t in (x, ga, gx, dy, A, ba, bx))
    (r, rr), (i, ii) = slopes(GA + BA), slopes(GX + BX)
    v = W * r
    a = np.exp(v)
    root = np.ones_like(a) if unit else np.sqrt(-np.expm1(2 * v))
    q = np.zeros_like(a) if unit else a * a / root
    y, my = ref.scan(X, GA, GX, W, BA, BX, unit=unit)
    hp, mp = (np.concatenate([np.zeros_like(p[:, :1]), p[:, :-1]], 1) for p in (y, my))
    lam, ml = DY.copy(), np.abs(DY)
    for t in range(L - 2, -1, -1):
        lam[:, t] += a[:, t + 1] * lam[:, t + 1]
        ml[:, t] += a[:, t + 1] * ml[:, t + 1]
    dv, mv = lam * (a * hp - q * i * X), ml * (a * (1 + np.abs(v) / 8) * mp + q * (1 + np.abs(v) / 4) * np.abs(i * X))
    # (r itself, of a shut gate, has the exponent's error too, and dv takes it through the root)
    sa, sx = 1 + np.abs(GA + BA) / 8, 1 + np.abs(GX + BX) / 8
    dga, ma = dv * W * rr, mv * np.abs(W) * rr * sa * sa
    dgx, mg = lam * root * X * ii, ml * root * np.abs(X) * ii * sx * sa
    lost = 2.0 ** -125  # of 1 - r
    fa, fx = mv * np.abs(W) * r * lost, ml * root * np.abs(X) * i * lost
    half = ref.HALF_STEP[dtype]
    both = (0, 1)
    for n, want, mag, floor in (("dgate_a", dga, ma, fa), ("dgate_x", dgx, mg, fx)):
        off = np.abs(f64(got[n]) - want) / (ref.bar(L) * mag + half * np.abs(want) + floor + 1e-37)
        assert off.max() <= 1, (n, off.max())
    for n, want, mag, floor in (("dbias_a", dga, ma, fa), ("dbias_x", dgx, mg, fx)):
        off = np.abs(f64(got[n]) - want.sum(both)) / (ref.bar(L) * mag.sum(both) + floor.sum(both) + 1e-37)
        assert off.max() <= 1, (n, off.max())


def test_gates_that_are_not_finite(torch_cuda):
    """An infinite gate is 0 or 1 with a slope of 0; a NaN is one in everything it enters."""
    from selective_state_space_63_amd import gated
    torch = torch_cuda
    b, L, d = 1, 10, 8
    g = np.random.default_rng(73)
    x, dy, ga, gx = (rows(torch, g, (b, L, d), "f32") for _ in range(4))
    A = -torch.full((d,), 0.3, device="cuda")
    inf = float("inf")
    ga[0, 4, 0], ga[0, 4, 1], gx[0, 4, 2], gx[0, 4, 3] = inf, -inf, inf, -inf
    ga[0, 4, 4], gx[0, 4, 5] = float("nan"), float("nan")
    out = gated.gated_scan_bwd(x, ga, gx, A, dy, unit_input=True)
    fine = [0, 1, 2, 3, 6, 7]
    assert all(bool(torch.isfinite(t[..., fine]).all()) for t in out.values())
    tiny = 2.0 ** -126
    assert bool((out["dgate_a"][0, 4, :2].abs() <= tiny).all()) and bool((out["dgate_x"][0, 4, 2:4].abs() <= tiny).all())
    assert float(out["dx"][0, 4, 3]) == 0
    assert bool(torch.isnan(out["dgate_a"][0, 4, 4])) and bool(torch.isnan(out["dA"][4]))
    assert bool(torch.isnan(out["dgate_x"][0, 4, 5])) and bool(torch.isnan(out["dx"][0, 4, 5]))


@pytest.mark.parametrize("which", ["x", "gate_a", "gate_x"])
@pytest.mark.parametrize("dim,step,dtype", [(66, 8, "bf16"), (66, 8, "f32"), (33, 7, "bf16"), (40, 1, "f32")])
@pytest.mark.parametrize("L", [5, 130])
def test_overlapping_rows_end_at_the_last_token(torch_cuda, L, dim, step, dtype, which):
    """Token rows closer than they are wide: what a tile's places past the last
    token would hold lies in the tensor, and enters nothing."""
    from selective_state_space_63_amd import gated
    torch = torch_cuda
    print(f"[case] overlapping rows {L} {dim} {step} {dtype} {which}", flush=True)
    g = np.random.default_rng([74, dim, L])
    k = {n: rows(torch, g, (1, L, dim), dtype) for n in ("x", "gate_a", "gate_x")}
    dy, A = rows(torch, g, (1, L, dim), dtype), -torch.from_numpy(g.uniform(0.05, 0.5, dim).astype(np.float32)).cuda()
    flat = rows(torch, g, ((L - 1) * step + dim,), dtype)
    at = dim // 2
    flat[(L - 1) * step + at] = float("nan")   # channel `at` of the last token
    k[which] = flat.as_strided((1, L, dim), (L * step, step, 1))
    zero = torch.zeros(dim, device="cuda")
    got = gated.gated_scan_bwd(**k, A=A, dy=dy, bias_a=zero, bias_x=zero)
    reads = torch.isnan(k[which]).any(1)[0]    # channels that hold the value at some token
    flat[(L - 1) * step + at] = 1.0            # (the same layout: rows that are whole may be summed in pairs)
    want = gated.gated_scan_bwd(**k, A=A, dy=dy, bias_a=zero, bias_x=zero)
    assert 0 < int(reads.sum()) < dim
    for n in got:
        assert bool(torch.isfinite(got[n][..., ~reads]).all()), n
        assert torch.equal(got[n][..., ~reads], want[n][..., ~reads]), n


@pytest.mark.parametrize("unit", [False, True], ids=["root", "unit"])
@pytest.mark.parametrize("dim,dtype", [(66, "bf16"), (33, "f32")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_gate_of_a_start_enters_nothing(torch_cuda, value, dim, dtype, unit):
    """At a start a = 0 and b = 1 whatever the gate holds: the bits of a gate of 0."""
    from selective_state_space_63_amd import gated
    torch = torch_cuda
    print(f"[case] gate of a start {value} {dim} {dtype} {unit}", flush=True)
    b, L = 2, 150
    g = np.random.default_rng([75, dim])
    x, dy, ga, gx = (rows(torch, g, (b, L, dim), dtype) for _ in range(4))
    A = -torch.from_numpy(g.uniform(0.05, 0.5, dim).astype(np.float32)).cuda()
    starts = torch.zeros(b, L, dtype=torch.bool, device="cuda")
    starts[0, [0, 60, 140]] = True
    starts[1, [5, 6, 149]] = True
    h0, zero = torch.ones(b, dim, device="cuda"), torch.zeros(dim, device="cuda")

    def call(fill):
        k = dict(x=x, gate_a=ga.masked_fill(starts[..., None], fill), gate_x=gx, A=A, bias_a=zero, bias_x=zero, h0=h0,
                 starts=starts, unit_input=unit)
        out = gated.gated_scan_bwd(**k, dy=dy)
        out["y"], out["h_last"] = gated.gated_scan_fwd(**k, return_last_state=True)
        return out

    want, got = call(0.0), call(value)
    for n in want:
        assert torch.equal(want[n], got[n]), n


@pytest.mark.parametrize("which", ["x", "gate_a", "gate_x"])
@pytest.mark.parametrize("step", [0, 8, (1 << 30) + 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_stride_of_a_single_token_is_not_read(torch_cuda, dtype, step, which):
    """One token of rows that overlap, or whose stride is past 32 bits of bytes."""
    from selective_state_space_63_amd import gated
    torch = torch_cuda
    print(f"[case] stride of a single token {step} {dtype} {which}", flush=True)
    dim = 66
    g = np.random.default_rng(76)
    k = {n: rows(torch, g, (1, 1, dim), dtype) for n in ("x", "gate_a", "gate_x")}
    dy, A = rows(torch, g, (1, 1, dim), dtype), -torch.from_numpy(g.uniform(0.05, 0.5, dim).astype(np.float32)).cuda()
    zero = torch.zeros(dim, device="cuda")
    k[which][0, 0, 40] = float("nan")
    want = gated.gated_scan_bwd(**k, A=A, dy=dy, bias_a=zero, bias_x=zero)
    k[which] = k[which].flatten().as_strided((1, 1, dim), (dim, step, 1))
    got = gated.gated_scan_bwd(**k, A=A, dy=dy, bias_a=zero, bias_x=zero)
    others = [c for c in range(dim) if c != 40]
    for n in want:
        assert bool(torch.isfinite(got[n][..., others]).all()), n
        assert torch.equal(got[n][..., others], want[n][..., others]), n
