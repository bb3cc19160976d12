"""Both kernels of the products with 4-bit weights (include/s6_q4.h), the slices
of the columns and every tile of rows among them, in the calls that a program
makes: a row that is not finite beside others, captured graphs, several streams."""
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


def operands(torch, m, k, n, group, dtype):
    g = np.random.default_rng([111, m, k, n])
    w = torch.from_numpy(g.integers(0, 256, (n, k // 2), dtype=np.uint8)).cuda()
    s = torch.from_numpy((0.02 * g.standard_normal((n, k // group))).astype(np.float32)).cuda().to(torch.bfloat16)
    x = torch.from_numpy(g.standard_normal((m, k)).astype(np.float32)).cuda()
    if dtype == "e4m3":
        xs = torch.from_numpy(g.uniform(0.5, 2, m).astype(np.float32)).cuda()
        return (20 * x).to(torch.float8_e4m3fn), xs, w, s
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32), None, w, s


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("m", [2, 6, 7, 16, 17, 20, 40, 130])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_not_finite_stays_in_its_row(torch_cuda, dtype, m, group):
    """Rows that hold a NaN or an infinity leave the bits of the others alone;
    8-bit rows as well with a factor that is not finite."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    print(f"[case] q4 rows not finite {m} {group} {dtype}", flush=True)
    x, xs, w, s = operands(torch, m, 256, 48, group, dtype)
    y = q4.q4_linear(x, w, s, x_scale=xs)
    bad = sorted({0, m // 2, m - 1} if m > 2 else {m - 1})
    xb = x.float()
    for i, t in enumerate(bad):
        xb[t, 37 * i + 5] = float("nan") if i % 2 == 0 or dtype == "e4m3" else float("inf")
    xb = xb.to(x.dtype)
    keep = [t for t in range(m) if t not in bad]
    yb = q4.q4_linear(xb, w, s, x_scale=xs)
    assert torch.equal(yb[keep], y[keep]) and not bool(torch.isfinite(yb[bad]).any())
    if xs is not None:
        xs = xs.clone()
        xs[bad[0]] = float("nan")
        xs[bad[-1]] = float("inf") if len(bad) > 1 else float("nan")
        yb = q4.q4_linear(x, w, s, x_scale=xs)
        assert torch.equal(yb[keep], y[keep]) and bool(torch.isnan(yb[bad[0]]).all())


CALLS = [
    # rows, inner, outer, group, dtype
    (6, 1024, 500, 128, "bf16"),      # few rows
    (25, 2560, 333, 128, "bf16"),     # slices of the columns
    (25, 2560, 333, 64, "e4m3"),
    (7, 2560, 333, 32, "f32"),        # slices, three parts
    (200, 512, 260, 128, "f32"),
    (256, 384, 8333, 128, "e4m3"),    # tiles of 96 rows on 256 CUs
    (384, 256, 10576, 32, "bf16"),    # of 64
]


@pytest.mark.parametrize("call", CALLS, ids=str)
def test_captured_and_replayed(torch_cuda, call):
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    print(f"[case] q4 graph {call}", flush=True)
    x, xs, w, s = operands(torch, *call)
    run = lambda: q4.q4_linear(x, w, s, x_scale=xs)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        if i == 2:
            x.copy_(x.float().neg().roll(1, 0).to(x.dtype))
        want = run()
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_two_graphs_share_nothing(torch_cuda):
    """Graphs captured one after another, replayed in either order."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    sets = [operands(torch, 25, 2560, n, 128, "bf16") for n in (333, 400)]
    want = [q4.q4_linear(x, w, s) for x, _, w, s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, _, w, s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(q4.q4_linear(x, w, s))
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert torch.equal(outs[i], want[i]), order


def test_two_streams(torch_cuda):
    """All of the kernels at once on two streams: the same bits every time."""
    from selective_state_space_63_amd import q4
    torch = torch_cuda
    sets = [operands(torch, *c) for c in CALLS]
    run = lambda: [q4.q4_linear(x, w, s, x_scale=xs) for x, xs, w, s in sets]  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
