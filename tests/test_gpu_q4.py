"""Products with 4-bit weights, their packing, and the norm with an 8-bit
output (include/s6_q4.h) against plain 64-bit references.

Bars.  Products: a sum of K exact products in fp32, in any order, is off by a
random walk of its roundings (one of 2^-24 of the running sum per term at most;
a few at every group, wave and row factor): 2^-24 (16 + sqrt(K)) of the sum of the
terms' absolute values; an fp32 x is there but for 2^-24 of it.  bf16 results one
rounding, 2^-8 of the value, besides.  Norm: 2^-18 of the magnitude, as the norms'
tests; the 8-bit value is the nearest one, half a step off at most, where the
step is 2^(e - 3) for values of exponent e, and 2^-9 below 2^-6.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
EPS = 1e-5


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_63_amd import s6
    s6.load_library()
    return torch


f64 = lambda t: None if t is None else t.detach().float().double().cpu().numpy()  # noqa: E731


def weights(torch, outer, inner, group, seed):
    """Codes at random (each value, zeros of both signs) and scales of either size."""
    g = np.random.default_rng([seed, outer, inner])
    w = torch.from_numpy(g.integers(0, 256, (outer, inner // 2), dtype=np.uint8)).cuda()
    s = torch.from_numpy((g.standard_normal((outer, inner // group)) * 0.02).astype(np.float32)).cuda().to(torch.bfloat16)
    return w, s


def unpack(w, s):
    c = w.cpu().numpy()
    v = VALUES[np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)]
    s = f64(s)
    return (v.reshape(*s.shape, -1) * s[..., None]).reshape(v.shape)


def rows(torch, m, k, dtype, seed, wide=0):
    g = np.random.default_rng([seed, m, k, 1])
    x = torch.from_numpy((2 * g.standard_normal((m, k + wide))).astype(np.float32)).cuda()
    if dtype == "e4m3":
        xs = torch.from_numpy(g.uniform(0.5, 2, m).astype(np.float32)).cuda()
        return (20 * x).clamp(-448, 448).to(torch.float8_e4m3fn)[:, wide:], xs
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)[:, wide:], None


def check(torch, x, xs, w, s, **kw):
    from selective_state_space_63_amd import q4
    y = q4.q4_linear(x, w, s, x_scale=xs, **kw)
    W, X = unpack(w, s), f64(x)
    if xs is not None:
        X = X * f64(xs)[:, None]
    want, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    got = f64(y)
    assert got.shape == want.shape and np.isfinite(got).all()
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    allowed = 2.0 ** -24 * (16 + math.sqrt(X.shape[1])) * mag + half * np.abs(want) + 1e-37
    worst = float(np.max(np.abs(got - want) / allowed)) if got.size else 0.0
    assert worst <= 1.0, f"{worst:.2f} of what is allowed"
    return y


SIZES = [
    # rows, inner, outer, group, columns before the slice of x
    (1, 32, 1, 32, 0),
    (1, 64, 16, 64, 0),
    (1, 128, 17, 128, 0),
    (2, 96, 33, 32, 8),
    (3, 192, 50, 64, 1),          # rows that 16-byte loads do not fit
    (6, 384, 40, 128, 0),
    (7, 1088, 99, 64, 0),
    (15, 2560, 130, 128, 0),
    (16, 1024, 257, 32, 0),
    (17, 640, 100, 128, 16),
    (24, 1664, 150, 64, 0),
    (25, 2560, 333, 128, 0),
    (32, 352, 130, 32, 5),
    (33, 8192, 20, 64, 0),
    (64, 256, 77, 128, 0),
    (65, 1152, 48, 32, 3),
    (130, 512, 200, 128, 0),
    (256, 384, 129, 128, 0),
    (300, 160, 64, 32, 0),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_products(torch_cuda, size, dtype):
    m, k, n, group, wide = size
    print(f"[case] q4 {size} {dtype}", flush=True)
    w, s = weights(torch_cuda, n, k, group, 51)
    x, xs = rows(torch_cuda, m, k, dtype, 52, wide)
    y = check(torch_cuda, x, xs, w, s)
    assert y.dtype == (torch_cuda.float32 if dtype == "f32" else torch_cuda.bfloat16)
    other = torch_cuda.bfloat16 if dtype == "f32" else torch_cuda.float32
    assert check(torch_cuda, x, xs, w, s, out_dtype=other).dtype == other
    if dtype == "e4m3":
        check(torch_cuda, x, None, w, s)


@pytest.mark.parametrize("size", [
    # where the tiles of rows are 96 high on 256 CUs: the last of 1 to 66 rows,
    # one and several blocks of columns; odd columns, rows that wide loads do not fit
    (256, 384, 8333, 128, 0),
    (258, 256, 8448, 64, 0),
    (193, 160, 10101, 32, 1),
    (1000, 288, 2560, 32, 0),
], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_products_of_many_tiles(torch_cuda, size, dtype):
    m, k, n, group, wide = size
    print(f"[case] q4 {size} {dtype}", flush=True)
    w, s = weights(torch_cuda, n, k, group, 61)
    x, xs = rows(torch_cuda, m, k, dtype, 62, wide)
    y = check(torch_cuda, x, xs, w, s)
    assert torch_cuda.equal(y, check(torch_cuda, x, xs, w, s))


def test_every_code_and_place(torch_cuda):
    """One column of x at a time is the column of the weights, exactly."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    for group, inner in ((128, 256), (64, 192), (32, 160)):
        w, s = weights(torch, 40, inner, group, 53)
        s.copy_(torch.exp2(torch.randint(-3, 4, s.shape, device="cuda").float()))
        W = unpack(w, s)
        for dt in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
            y = q4.q4_linear(torch.eye(inner, device="cuda").to(dt), w, s, out_dtype=torch.float32)
            assert np.array_equal(f64(y), W.T), (group, dt)


def test_fp32_rows_enter_in_full(torch_cuda):
    """Values that bf16 would round away, of sizes far apart."""
    torch = torch_cuda
    w, s = weights(torch, 64, 256, 128, 54)
    g = np.random.default_rng(55)
    x = torch.from_numpy((g.standard_normal((5, 256)) * 10.0 ** g.uniform(-6, 6, (5, 256))).astype(np.float32)).cuda()
    check(torch, x, None, w, s)
    check(torch, x * 1e-25, None, w, s)


@pytest.mark.parametrize("m", [1, 20, 40])
@pytest.mark.parametrize("group", [32, 128])
def test_largest_fp32_values(torch_cuda, m, group):
    """Values that bf16 would round to infinity are finite, and stay so."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    print(f"[case] q4 largest fp32 {m} {group}", flush=True)
    w = torch.full((48, 64), 0x11, dtype=torch.uint8, device="cuda")  # 0.5
    s = torch.full((48, 128 // group), 2.0 ** -6, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(m, 128, device="cuda")
    x[0, 0], x[-1, 127] = 3.4e38, -3.4028234e38
    check(torch, x, None, w, s)
    x[0, 3], x[-1, 5] = float("inf"), float("nan")
    y = q4.q4_linear(x, w, s)
    if m > 1:
        assert bool(torch.isinf(y[0]).all()) and bool(torch.isfinite(y[1:-1]).all())
    assert bool(torch.isnan(y[-1]).all())


def test_not_finite_stays_in_its_row(torch_cuda):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    for group in (32, 128):
        w, s = weights(torch, 48, 256, group, 56)
        for dt in (torch.bfloat16, torch.float32):
            x = torch.randn(20, 256, device="cuda").to(dt)
            y = q4.q4_linear(x, w, s)
            bad = x.clone()
            bad[3, 7], bad[5, 200], bad[17, 64] = float("nan"), float("inf"), -float("inf")
            yb = q4.q4_linear(bad, w, s)
            keep = [t for t in range(20) if t not in (3, 5, 17)]
            assert torch.equal(yb[keep], y[keep]) and not bool(torch.isfinite(yb[[3, 5, 17]]).any())


def test_empty_and_shapes(torch_cuda):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    w, s = weights(torch, 24, 128, 64, 57)
    assert q4.q4_linear(torch.zeros(0, 128, device="cuda"), w, s).shape == (0, 24)
    assert q4.q4_linear(torch.zeros(3, 128, device="cuda"), w[:0], s[:0]).shape == (3, 0)
    x = torch.randn(2, 3, 128, device="cuda")
    y = q4.q4_linear(x, w, s)
    assert torch.equal(y.flatten(0, 1), q4.q4_linear(x.flatten(0, 1), w, s))
    v = q4.q4_linear(x[0, 0], w, s)
    assert v.shape == (24,) and torch.equal(v, q4.q4_linear(x[0, :1], w, s)[0])
    out = torch.empty(2, 3, 24, device="cuda")
    assert q4.q4_linear(x, w, s, y=out) is out and torch.equal(out, y)


@pytest.mark.parametrize("shape", [(1, 32, 32), (7, 96, 32), (33, 128, 64), (50, 256, 128), (300, 2560, 128)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pack(torch_cuda, shape, dtype):
    """Scales and codes are the nearest ones, ties to the even code."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    n, k, group = shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    w = torch.from_numpy(np.random.default_rng([58, n, k]).standard_normal((n, k + 3)).astype(np.float32)).cuda().to(dt)[:, 3:]
    w[0, :32] = 0
    codes, scales = q4.q4_pack(w, group)
    v = w.float().cpu().numpy().reshape(n, -1, group)
    top = torch.from_numpy(np.abs(v).max(-1) / np.float32(6))
    assert torch.equal(scales.cpu(), top.to(torch.bfloat16))
    sc = scales.float().cpu().numpy()[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(sc > 0, v / sc, np.float32(0)).astype(np.float32)   # fp32, as documented: w / scale
    c = codes.cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(t.shape)
    off = np.abs(VALUES[c] - t)
    best = np.abs(VALUES[:, None, None, None] - t[None]).min(0)
    # (a largest value may lie past 6, by the rounding of the scale)
    assert (off <= best * (1 + 1e-6) + 1e-12).all()
    tie = np.isin(np.abs(t), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert (c[tie] % 2 == 0).all()


def test_pack_ties(torch_cuda):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    w = torch.zeros(1, 32, device="cuda")
    w[0, :15] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
    c, s = q4.q4_pack(w, 32)
    c = c.cpu().numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(-1)
    assert float(s[0, 0]) == 1.0
    assert np.array_equal(VALUES[c[:15]], [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4]) and not c[15:].any()


def test_pack_of_what_is_not_finite(torch_cuda):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    w = torch.randn(2, 128, device="cuda")
    w[0, 40], w[1, 3] = float("nan"), float("inf")
    c, s = q4.q4_pack(w, 32)
    fine = torch.isfinite(s)
    assert not bool(fine[0, 1]) and not bool(fine[1, 0]) and int(fine.sum()) == 6


ADD = [
    # rows, dim, dtype, residual dtype (None: no residual), gamma, extra columns
    (1, 1, "f32", "f32", True, 0),
    (1, 8, "bf16", "f32", False, 0),
    (5, 7, "bf16", "bf16", True, 0),
    (3, 64, "bf16", None, True, 0),
    (600, 520, "bf16", "bf16", True, 8),
    (33, 2048, "bf16", "f32", True, 0),
    (9, 2560, "bf16", "f32", True, 3),      # rows that 16-byte loads do not fit
    (5, 2047, "f32", "f32", True, 0),
    (4, 8200, "bf16", "f32", True, 0),      # wider than the registers
    (2, 20000, "f32", None, True, 0),
    (3000, 1100, "bf16", "f32", False, 1),  # several rows per workgroup
    (5000, 64, "f32", "f32", True, 0),
]


@pytest.mark.parametrize("shape", ADD, ids=str)
def test_add_norm_q8(torch_cuda, shape):
    from selective_state_space_63_amd import block, q4
    torch = torch_cuda
    m, dim, dtype, rd, has_gamma, wide = shape
    print(f"[case] add norm q8 {shape}", flush=True)
    g = np.random.default_rng([59, m, dim])
    ty = dict(bf16=torch.bfloat16, f32=torch.float32)
    put = lambda a, d: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(ty[d])  # noqa: E731
    x = put(3 * g.standard_normal((m, dim + wide)), dtype)[:, wide:]
    r = None if rd is None else put(2 * g.standard_normal((m, dim)), rd)
    w = put(1 + 0.3 * g.standard_normal(dim), "f32")
    gm = put(g.standard_normal(dim), "f32") if has_gamma else None
    args = dict(residual=r, gamma=gm, scale=0.6, eps=EPS)
    out, sc, res = q4.add_norm_q8_fwd(x, w, **args)
    assert out.dtype == torch.float8_e4m3fn and sc.shape == (m,)
    # the residual has the bits of add_norm_fwd's
    plain, want_res = block.add_norm_fwd(x, w, **args)
    assert torch.equal(res, want_res)
    k = np.float64(np.float32(0.6)) * (1.0 if gm is None else f64(gm))
    rr = k * f64(x) + (0.0 if r is None else f64(r))
    o = rr / np.sqrt((rr * rr).mean(-1, keepdims=True) + EPS) * f64(w)
    top = np.abs(o).max(-1)
    # r' is off by the roundings of its two terms
    mag = (np.abs(k * f64(x)) + (0.0 if r is None else np.abs(f64(r)))) * np.abs(f64(w)) / np.sqrt((rr * rr).mean(-1, keepdims=True) + EPS)
    assert (np.abs(f64(sc) - top / 448) <= 2.0 ** -18 * mag.max(-1) / 448).all()
    v = o / f64(sc)[:, None]
    code = f64(out)
    assert np.abs(code).max() == 448
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    off = np.abs(code - v) - (2.0 ** (e - 4) + 2.0 ** -17 * (np.abs(v) + mag / f64(sc)[:, None]))
    assert (off <= 0).all()
    # in place on the residual, the same bits; every call the same bits
    if r is not None:
        out2, sc2, res2 = q4.add_norm_q8_fwd(x, w, residual_out=r, **args)
        assert res2 is r and torch.equal(r, want_res)
        assert torch.equal(out.view(torch.uint8), out2.view(torch.uint8)) and torch.equal(sc, sc2)


def test_add_norm_q8_rows_of_nothing_and_not_finite(torch_cuda):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    for dim in (64, 1000, 2560, 20000):
        x = torch.randn(8, dim, device="cuda")
        x[1] = 0
        x[2] *= 1e-36            # squares vanish beside eps, outputs are below 2^-100
        x[3, dim // 2] = float("nan")
        x[4, 5] = float("inf")
        w = torch.ones(dim, device="cuda")
        out, sc, _ = q4.add_norm_q8_fwd(x, w, eps=EPS)
        o = out.float()
        for t in (1, 2):
            assert float(sc[t]) == 0 and not bool(o[t].any())
        for t in (3, 4):
            assert bool(torch.isnan(sc[t])) and bool(torch.isnan(o[t]).all())
        fine = [0, 5, 6, 7]
        assert bool(torch.isfinite(o[fine]).all()) and bool((sc[fine] > 0).all())
        w[7] = float("nan")
        out, sc, _ = q4.add_norm_q8_fwd(x, w, eps=EPS)
        assert bool(torch.isnan(sc).all()) and bool(torch.isnan(out.float()).all())
    e = q4.add_norm_q8_fwd(torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda"))
    assert e[0].shape == (0, 64) and e[1].shape == (0,)


@pytest.mark.parametrize("largest", [2.0 ** -99, 1e-20, 1e30, 2.0 ** 127])
def test_add_norm_q8_of_any_size(torch_cuda, largest):
    """Rows of +-1: outputs are the weight's size, stored as 448 of
    the scale, whatever that size is."""
    from selective_state_space_63_amd import q4
    print(f"[case] add_norm_q8 largest {largest}", flush=True)
    g = np.random.default_rng(81)
    x = torch_cuda.from_numpy(g.choice([-1.0, 1.0], (3, 64)).astype(np.float32)).cuda()
    w = torch_cuda.full((64,), largest, dtype=torch_cuda.float32, device="cuda")
    out, scale, _ = q4.add_norm_q8_fwd(x, w, eps=0.0)
    assert torch_cuda.equal(out.float(), 448 * x)
    assert float((scale.double() * 448 / largest - 1).abs().max()) <= 2.0 ** -18


def test_norm_then_products(torch_cuda):
    """The two as they are used: rows in 8 bits with their factors go into the
    products; against the products of the norm's own output the result is off by
    the 8-bit rounding, half a step of each value at most."""
    from selective_state_space_63_amd import block, q4
    torch = torch_cuda
    g = torch.Generator("cuda").manual_seed(60)
    for m in (1, 4, 40, 200):
        x = torch.randn(m, 640, device="cuda", generator=g).to(torch.bfloat16)
        r = torch.randn(m, 640, device="cuda", generator=g)
        nw = 1 + 0.1 * torch.randn(640, device="cuda", generator=g)
        w, s = q4.q4_pack(torch.randn(300, 640, device="cuda", generator=g) / 25)
        q, sc, r1 = q4.add_norm_q8_fwd(x, nw, residual=r)
        y = check(torch, q, sc, w, s, out_dtype=torch.float32)
        o, r2 = block.add_norm_fwd(x.float(), nw, residual=r)
        assert torch.equal(r1, r2)
        W, X, Q = unpack(w, s), f64(o), f64(q)
        step = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(Q), 2.0 ** -6))) - 4), 2.0 ** -10) * f64(sc)[:, None]
        assert (np.abs(f64(y) - X @ W.T) <= 1.01 * step @ np.abs(W).T + 2.0 ** -16 * np.abs(X) @ np.abs(W).T).all()


def test_graph_and_streams(torch_cuda):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    w, s = weights(torch, 500, 1024, 128, 61)
    nw = torch.ones(1024, device="cuda")
    x, r = torch.randn(6, 1024, device="cuda").to(torch.bfloat16), torch.randn(6, 1024, device="cuda")

    def run():
        q, sc, res = q4.add_norm_q8_fwd(x, nw, residual=r)
        return q4.q4_linear(q, w, s, x_scale=sc), q4.q4_linear(x, w, s), res

    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        if i == 2:
            x.mul_(-1.5)
        want = run()
        torch.cuda.synchronize()
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_many_rows_and_large_weights(torch_cuda):
    """Rows past one launch, and codes past 2^31 bytes."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    w, s = weights(torch, 5, 32, 32, 62)
    m = 65535 * 16 + 40
    x = torch.randn(m, 32, device="cuda").to(torch.bfloat16)
    y = q4.q4_linear(x, w, s, out_dtype=torch.float32)
    W = torch.from_numpy(unpack(w, s)).cuda()
    want = x.double() @ W.t().contiguous()
    mag = x.double().abs() @ W.abs().t().contiguous()
    assert bool(((y.double() - want).abs() <= 2.0 ** -24 * (16 + math.sqrt(32)) * mag).all())
    n, k = 1_100_000, 4096
    w = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    s = torch.ones(n, k // 128, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, k, device="cuda").to(torch.bfloat16)
    y = q4.q4_linear(x, w, s, out_dtype=torch.float32)
    tail = check(torch, x, None, w[-50:].contiguous(), s[-50:].contiguous(), out_dtype=torch.float32)
    assert torch.equal(y[:, -50:], tail)
