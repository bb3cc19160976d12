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


def test_gradients_that_nobody_asks_for_are_not_taken(torch_cuda):
    """Without a residual, AddNorm's backward makes no residual's gradient (the
    largest tensor of it); weights that are not trained get none."""
    from selective_state_space_63_amd import block
    torch = torch_cuda
    rows, dim = 4096, 2048
    x = torch.randn(rows, dim, device="cuda").to(torch.bfloat16).requires_grad_()
    w = torch.ones(dim, device="cuda")
    out, _ = block.AddNorm.apply(x, w)
    dout = torch.randn_like(out)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    dx, = torch.autograd.grad(out, x, dout)
    # dx, and room for the column sums' parts that the query asks for
    assert torch.cuda.max_memory_allocated() - before <= 2 * rows * dim + 2 * 1024 * dim * 4 + (1 << 20)
    del dx
    g = torch.Generator("cuda").manual_seed(72)
    y, z, r = (torch.randn(50, 64, device="cuda", generator=g) for _ in range(3))
    w, gm = (torch.randn(64, device="cuda", generator=g) for _ in range(2))
    do = torch.randn(50, 64, device="cuda", generator=g)
    for fn, args in ((block.AddNorm, (y, w, r, gm, 0.5)), (block.GatedNorm, (y, z, w, 2))):
        names = [i for i, a in enumerate(args) if torch.is_tensor(a)]
        full = [a.clone().requires_grad_() if i in names else a for i, a in enumerate(args)]
        res = fn.apply(*full)
        all_ = torch.autograd.grad(res if torch.is_tensor(res) else res[0], [full[i] for i in names], do)
        for i, want in zip(names, all_):  # each alone, the same bits
            one = [a.clone().requires_grad_() if j == i else a for j, a in enumerate(args)]
            res = fn.apply(*one)
            got, = torch.autograd.grad(res if torch.is_tensor(res) else res[0], one[i], do)
            assert torch.equal(got, want), (fn, i)
    d = heads_inputs(torch)
    names = ("x", "delta", "A", "Bm", "Cm", "D", "h0", "bias")
    dy = torch.randn_like(d["x"])
    full = [d[k].clone().requires_grad_() for k in names]
    all_ = torch.autograd.grad(block.HeadsScan.apply(*full, True, False)[0], full, dy)
    for i, want in enumerate(all_):
        one = [d[k].clone().requires_grad_() if j == i else d[k] for j, k in enumerate(names)]
        got, = torch.autograd.grad(block.HeadsScan.apply(*one, True, False)[0], one[i], dy)
        assert torch.equal(got, want), names[i]


def test_tensors_written_in_place_are_marked(torch_cuda):
    """A backward that saved a state, a residual or an output buffer refuses it
    after a call has written there, as with torch's own in-place operations;
    tensors of inference mode have nothing to mark and are taken as before."""
    from selective_state_space_63_amd import block
    torch = torch_cuda
    d = heads_inputs(torch)
    w = torch.ones(64, device="cuda")

    def saved(t, call):
        p = torch.ones_like(t, requires_grad=True)
        loss = (t * p).sum()  # keeps t for p's gradient
        call(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()

    one = [d[k][:, 0].contiguous() for k in ("x", "delta")] + [d["A"]] + [d[k][:, 0].contiguous() for k in ("Bm", "Cm")]
    seq = [d[k] for k in ("x", "delta", "A", "Bm", "Cm")]
    rows = torch.randn(5, 64, device="cuda")
    saved(d["h0"].clone(), lambda t: block.heads_state_update(t, *one))
    saved(torch.zeros_like(one[0]), lambda t: block.heads_state_update(d["h0"].clone(), *one, y=t))
    saved(torch.zeros_like(d["x"]), lambda t: block.heads_scan_fwd(*seq, y=t))
    saved(torch.zeros_like(d["h0"]), lambda t: block.heads_scan_fwd(*seq, h_last=t))
    saved(rows.clone(), lambda t: block.add_norm_fwd(rows, w, residual=t, residual_out=t))
    saved(rows.clone(), lambda t: block.add_norm_fwd(rows, w, out=t))
    saved(rows.clone(), lambda t: block.gated_norm_fwd(rows, rows, w, out=t))
    with torch.inference_mode():
        h = d["h0"].clone()
    want = d["h0"].clone()
    block.heads_state_update(h, *one)
    block.heads_state_update(want, *one)
    assert torch.equal(h, want)
