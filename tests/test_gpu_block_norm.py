"""The norms before and after a block (include/s6_block.h) against the plain
64-bit reference.

Bars: fp32 results are within a few dozen roundings of their terms (row sums
over register pieces and a tree of threads, v_rsq_f32 and v_rcp_f32 to one
unit, the exponential of a gate to a few): 2^-18 of the magnitude; column sums
over up to 600 rows the same.  Results rounded to bf16: 2^-8 (one rounding is
2^-9, and the magnitude bounds the value).
"""
import numpy as np
import pytest

import block_ref as ref

pytestmark = pytest.mark.gpu

F32_BAR, BF16_BAR, EPS = 2.0 ** -18, 2.0 ** -8, 1e-5


@pytest.fixture(scope="module")
def torch_cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from selective_state_space_63_amd import s6
    s6.load_library()
    return torch


def close(got, want, mag, what):
    bound = BF16_BAR if "bfloat16" in str(got.dtype) else F32_BAR
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = float(np.max(np.abs(got - want) / np.maximum(mag, 1e-30))) if got.size else 0.0
    assert worst <= bound, f"{what}: {worst:.3e} of the magnitude, bar {bound:.3e}"


def put(torch, a, dtype, wide=0):
    """On the device, as a slice of rows `wide` elements wider."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    t = t.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    if wide:
        full = torch.zeros(*t.shape[:-1], t.shape[-1] + wide, dtype=t.dtype, device="cuda")
        full[..., :t.shape[-1]] = t
        return full[..., :t.shape[-1]]
    return t


f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731

ADD = [
    # rows, dim, dtype, residual dtype (None: no residual), gamma, wide
    (1, 1, "f32", "f32", True, 0),
    (1, 8, "bf16", "f32", False, 0),
    (5, 7, "bf16", "bf16", True, 0),
    (3, 64, "bf16", None, True, 0),
    (600, 520, "bf16", "bf16", True, 8),
    (33, 2048, "bf16", "f32", True, 0),
    (17, 2056, "f32", "f32", False, 0),
    (9, 2560, "bf16", "f32", True, 3),      # rows that 16-byte loads do not fit
    (5, 2047, "f32", "f32", True, 0),
    (4, 8200, "bf16", "f32", True, 0),      # wider than the registers
    (2, 20000, "f32", None, True, 0),
    (3, 1100, "bf16", "f32", True, 1),
]


@pytest.mark.parametrize("shape", ADD, ids=str)
def test_add_norm(torch_cuda, shape):
    from selective_state_space_63_amd import block
    torch = torch_cuda
    rows, dim, dtype, rd, has_gamma, wide = shape
    print(f"[case] add norm {shape}", flush=True)
    g = np.random.default_rng([21, rows, dim])
    x = put(torch, 3 * g.standard_normal((rows, dim)), dtype, wide)
    r = None if rd is None else put(torch, 2 * g.standard_normal((rows, dim)), rd)
    w = put(torch, 1 + 0.3 * g.standard_normal(dim), "f32")
    gm = put(torch, g.standard_normal(dim), "f32") if has_gamma else None
    out, res = block.add_norm_fwd(x, w, residual=r, gamma=gm, scale=0.6, eps=EPS)
    assert out.dtype == x.dtype and res.dtype == (torch.float32 if rd is None else r.dtype)
    ro, rr = ref.add_norm(f64(x), f64(r), f64(w), f64(gm), np.float32(0.6).astype(np.float64), EPS)
    k = 0.6 * (1.0 if gm is None else np.abs(f64(gm)))
    mr = k * np.abs(f64(x)) + (0.0 if r is None else np.abs(f64(r)))
    inv = np.abs(ro) / np.maximum(np.abs(rr * f64(w)), 1e-30)
    close(res, rr, mr, "residual")
    close(out, ro, mr * inv * np.abs(f64(w)) + np.abs(ro), "out")
    # in place on the residual, the same bits
    if r is not None:
        out2, res2 = block.add_norm_fwd(x, w, residual=r, gamma=gm, scale=0.6, eps=EPS, residual_out=r)
        assert res2 is r and torch.equal(out, out2) and torch.equal(res, r)

    do = put(torch, g.standard_normal((rows, dim)), dtype)
    dr = put(torch, g.standard_normal((rows, dim)), "f32").to(res.dtype)
    for dres in (dr, None):
        got = block.add_norm_bwd(do, res, w, dresidual_out=dres, x=x, gamma=gm, scale=0.6, eps=EPS)
        du, mdu, dw, mdw = ref.rms_bwd(f64(res), f64(do), f64(w), 1, EPS)
        if dres is not None:
            du, mdu = du + f64(dres), mdu + np.abs(f64(dres))
        kk = 0.6 * (np.ones(dim) if gm is None else f64(gm))
        close(got["dresidual"], du, mdu, "dresidual")
        close(got["dx"], du * kk, mdu * np.abs(kk), "dx")
        close(got["dweight"], dw, mdw, "dweight")
        assert ("dgamma" in got) == has_gamma
        if has_gamma:
            close(got["dgamma"], 0.6 * (du * f64(x)).sum(0), 0.6 * (mdu * np.abs(f64(x))).sum(0), "dgamma")


GATE = [
    # rows, dim, groups, dtype, after, gate, wide
    (1, 1, 1, "f32", False, True, 0),
    (3, 24, 3, "bf16", True, True, 0),
    (7, 21, 3, "bf16", False, True, 0),
    (600, 512, 1, "bf16", False, True, 8),
    (50, 2048, 8, "bf16", True, True, 0),
    (11, 5120, 1, "bf16", False, True, 64),
    (5, 5120, 2, "f32", True, True, 0),
    (9, 1544, 8, "f32", False, True, 5),
    (4, 9000, 1, "bf16", True, True, 0),     # wider than the registers
    (3, 4200, 2, "f32", False, True, 1),
    (6, 640, 1, "bf16", False, False, 0),    # no gate
]


@pytest.mark.parametrize("shape", GATE, ids=str)
def test_gated_norm(torch_cuda, shape):
    from selective_state_space_63_amd import block
    torch = torch_cuda
    rows, dim, groups, dtype, after, gate, wide = shape
    print(f"[case] gated norm {shape}", flush=True)
    g = np.random.default_rng([22, rows, dim])
    y = put(torch, 2 * g.standard_normal((rows, dim)), dtype, wide)
    z = put(torch, 2 * g.standard_normal((rows, dim)), dtype, 2 * wide) if gate else None
    w = put(torch, 1 + 0.3 * g.standard_normal(dim), "f32")
    out = block.gated_norm_fwd(y, z, w, groups=groups, gate_after=after, eps=EPS)
    ro = ref.gated_norm(f64(y), f64(z), f64(w), groups, after, EPS)
    close(out, ro, np.abs(ro), "out")
    do = put(torch, g.standard_normal((rows, dim)), dtype)
    got = block.gated_norm_bwd(do, y, z, w, groups=groups, gate_after=after, eps=EPS)
    yv, d = f64(y), f64(do)
    if gate:
        sg = 1 / (1 + np.exp(-f64(z)))
        f, df, mdf = f64(z) * sg, sg * (1 + f64(z) * (1 - sg)), sg * (1 + np.abs(f64(z)) * (1 - sg))
    else:
        f, df, mdf = np.ones_like(yv), None, None
    if after:
        du, mdu, dw, mdw = ref.rms_bwd(yv, d * f, f64(w), groups, EPS)
        dz = None if z is None else (d * ref.rms(yv, groups, EPS) * f64(w))
        mdz = None if z is None else np.abs(dz)
    else:
        du, mdu, dw, mdw = ref.rms_bwd(yv * f, d, f64(w), groups, EPS)
        dz, mdz = du * yv, mdu * np.abs(yv)
        du, mdu = du * f, mdu * np.abs(f)
    close(got["dy"], du, mdu, "dy")
    close(got["dweight"], dw, mdw, "dweight")
    assert ("dz" in got) == gate
    if gate:
        close(got["dz"], dz * df, mdz * mdf, "dz")


def test_gradients_against_differences(torch_cuda):
    """Both norms' fp32 gradients against central differences of the 64-bit
    forward along random directions (step 1e-5: exact to about 1e-9)."""
    from selective_state_space_63_amd import block
    torch = torch_cuda
    g = np.random.default_rng(23)
    rows, dim = 6, 40
    v = {k: g.standard_normal((rows, dim)).astype(np.float32) for k in ("x", "r", "z", "do", "dr")}
    v.update(w=g.standard_normal(dim).astype(np.float32), gm=g.standard_normal(dim).astype(np.float32))
    n = {k: a.astype(np.float64) for k, a in v.items()}
    t = {k: torch.from_numpy(a).cuda() for k, a in v.items()}
    out, res = block.add_norm_fwd(t["x"], t["w"], residual=t["r"], gamma=t["gm"], scale=0.5, eps=EPS)
    ga = block.add_norm_bwd(t["do"], res, t["w"], dresidual_out=t["dr"], x=t["x"], gamma=t["gm"], scale=0.5, eps=EPS)

    def add(u):
        o, r = ref.add_norm(u["x"], u["r"], u["w"], u["gm"], 0.5, EPS)
        return (o * n["do"]).sum() + (r * n["dr"]).sum()

    def check(loss, pairs):
        for k, grad in pairs:
            dirn, h = g.choice([-1.0, 1.0], n[k].shape), 1e-5
            diff = (loss({**n, k: n[k] + h * dirn}) - loss({**n, k: n[k] - h * dirn})) / (2 * h)
            own = grad.double().cpu().numpy()
            assert abs((own * dirn).sum() - diff) <= 2.0 ** -16 * np.abs(own).sum() + 1e-6, k

    check(add, (("x", ga["dx"]), ("r", ga["dresidual"]), ("w", ga["dweight"]), ("gm", ga["dgamma"])))
    for after in (False, True):
        gg = block.gated_norm_bwd(t["do"], t["x"], t["z"], t["w"], groups=4, gate_after=after, eps=EPS)
        check(lambda u: (ref.gated_norm(u["x"], u["z"], u["w"], 4, after, EPS) * n["do"]).sum(),
              (("x", gg["dy"]), ("z", gg["dz"]), ("w", gg["dweight"])))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan"), 3.0e38])
def test_rows_are_apart(torch_cuda, value):
    """A row with a value that is not finite, or whose square is not, leaves
    the other rows alone; a row of zeros gives zeros."""
    from selective_state_space_63_amd import block
    torch = torch_cuda
    x = torch.randn(6, 256, device="cuda")
    x[4] = 0.0
    w = torch.randn(256, device="cuda")
    z = torch.randn_like(x)
    clean = [block.add_norm_fwd(x, w)[0], block.gated_norm_fwd(x, z, w)]
    x[2, 17] = value
    dirty = [block.add_norm_fwd(x, w)[0], block.gated_norm_fwd(x, z, w)]
    keep = [0, 1, 3, 4, 5]
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
        assert torch.equal(b[4], torch.zeros_like(b[4]))


def test_gate_limits(torch_cuda):
    """SiLU at 0 and far out: 0 at 0, z at +large, 0 at -large, no NaN."""
    from selective_state_space_63_amd import block
    torch = torch_cuda
    y = torch.ones(1, 8, device="cuda")
    z = torch.tensor([[0.0, 200.0, -200.0, 3.0e38, -3.0e38, 1.0, -1.0, 50.0]], device="cuda")
    w = torch.ones(8, device="cuda")
    out = block.gated_norm_fwd(y, z, w, gate_after=True, eps=0.0)
    assert torch.isfinite(out).all()
    assert float(out[0, 0]) == 0.0 and abs(float(out[0, 1]) - 200) < 1e-3 and abs(float(out[0, 2])) < 1e-30
    g = block.gated_norm_bwd(torch.ones_like(y), y, z, w, gate_after=True, eps=1e-5)
    assert all(bool(torch.isfinite(v).all()) for v in g.values())
    assert abs(float(g["dz"][0, 0]) - 0.5) < 1e-4


def test_no_rows(torch_cuda):
    from selective_state_space_63_amd import block
    torch = torch_cuda
    x, w = torch.empty(0, 16, device="cuda"), torch.ones(16, device="cuda")
    out, res = block.add_norm_fwd(x, w)
    assert out.shape == (0, 16) and res.shape == (0, 16)
    g = block.add_norm_bwd(out, res, w, x=x, gamma=w)
    assert torch.equal(g["dweight"], torch.zeros(16, device="cuda")) and torch.equal(g["dgamma"], g["dweight"])
    assert block.gated_norm_fwd(x, x, w).shape == (0, 16)
    assert torch.equal(block.gated_norm_bwd(x, x, x, w)["dweight"], torch.zeros(16, device="cuda"))


def test_leading_dimensions_and_autograd(torch_cuda):
    from selective_state_space_63_amd import block
    torch = torch_cuda
    wide = torch.randn(3, 5, 72, device="cuda", dtype=torch.bfloat16)
    x, z = wide[..., :32], wide[..., 40:72]
    w = torch.randn(32, device="cuda", requires_grad=True)
    gm = torch.randn(32, device="cuda", requires_grad=True)
    a, b = x.detach().clone().requires_grad_(), z.detach().clone().requires_grad_()
    out, res = block.AddNorm.apply(a, w, None, gm, 0.5)
    assert torch.equal(out, block.add_norm_fwd(x, w.detach(), gamma=gm.detach(), scale=0.5)[0])
    o2 = block.GatedNorm.apply(out, b, w, 2, False)
    o2.float().sum().backward()
    ones = torch.ones_like(o2)
    g2 = block.gated_norm_bwd(ones, out.detach(), z, w.detach(), groups=2)
    g1 = block.add_norm_bwd(g2["dy"], res.detach(), w.detach(), x=x, gamma=gm.detach(), scale=0.5)
    assert torch.equal(a.grad, g1["dx"]) and torch.equal(b.grad, g2["dz"]) and torch.equal(gm.grad, g1["dgamma"])
    assert torch.allclose(w.grad, g1["dweight"] + g2["dweight"])
