"""The norms with more rows than a launch has row walkers (1024 where
column sums are taken, up to 8192 otherwise), so that a walker takes several
rows and the last turn is partial.

Bars as in test_gpu_block_norm.py: fp32 results 2^-18 of the magnitude.  A
column sum here adds up to 9 rows per walker, 16 walkers per thread and a tree
of 6, each term after about a dozen roundings: 43 * 2^-24 = 0.67 * 2^-18.
"""
import numpy as np
import pytest

import block_ref as ref
from test_gpu_block_norm import EPS, close, f64, put, torch_cuda  # noqa: F401

pytestmark = pytest.mark.gpu

ADD = [
    # rows, dim, dtype, residual dtype, gamma, wide
    (9001, 64, "bf16", "f32", True, 0),      # a wave per row
    (9001, 65, "f32", "f32", True, 0),       # (single values)
    (5003, 520, "bf16", "bf16", True, 8),    # a workgroup per row
    (4099, 1030, "f32", "f32", True, 3),     # (single values)
    (2100, 8200, "bf16", "f32", True, 0),    # wider than the registers
    (1500, 4200, "bf16", "bf16", True, 1),   # (single values)
]


@pytest.mark.parametrize("shape", ADD, ids=str)
def test_add_norm_turns(torch_cuda, shape):
    from selective_state_space_63_amd import block
    torch = torch_cuda
    rows, dim, dtype, rd, _, wide = shape
    print(f"[case] add norm {shape}", flush=True)
    g = np.random.default_rng([51, rows, dim])
    x = put(torch, 3 * g.standard_normal((rows, dim)), dtype, wide)
    r = put(torch, 2 * g.standard_normal((rows, dim)), rd)
    w, gm = (put(torch, 1 + 0.3 * g.standard_normal(dim), "f32") for _ in range(2))
    out, res = block.add_norm_fwd(x, w, residual=r, gamma=gm, scale=0.6, eps=EPS)
    ro, rr = ref.add_norm(f64(x), f64(r), f64(w), f64(gm), np.float32(0.6).astype(np.float64), EPS)
    mr = 0.6 * np.abs(f64(gm)) * np.abs(f64(x)) + np.abs(f64(r))
    inv = np.abs(ro) / np.maximum(np.abs(rr * f64(w)), 1e-30)
    close(res, rr, mr, "residual")
    close(out, ro, mr * inv * np.abs(f64(w)) + np.abs(ro), "out")
    do = put(torch, g.standard_normal((rows, dim)), dtype)
    dr = put(torch, g.standard_normal((rows, dim)), "f32").to(res.dtype)
    got = block.add_norm_bwd(do, res, w, dresidual_out=dr, x=x, gamma=gm, scale=0.6, eps=EPS)
    du, mdu, dw, mdw = ref.rms_bwd(f64(res), f64(do), f64(w), 1, EPS)
    du, mdu = du + f64(dr), mdu + np.abs(f64(dr))
    k = 0.6 * f64(gm)
    close(got["dresidual"], du, mdu, "dresidual")
    close(got["dx"], du * k, mdu * np.abs(k), "dx")
    close(got["dweight"], dw, mdw, "dweight")
    close(got["dgamma"], 0.6 * (du * f64(x)).sum(0), 0.6 * (mdu * np.abs(f64(x))).sum(0), "dgamma")


GATE = [
    # rows, dim, groups, dtype, after, wide
    (9001, 128, 2, "bf16", False, 0),        # a wave per row
    (9001, 63, 3, "f32", True, 0),           # (single values)
    (5003, 1040, 1, "bf16", True, 8),        # a workgroup per row
    (2500, 2060, 2, "f32", False, 3),        # (single values)
    (2100, 8200, 1, "bf16", False, 0),       # wider than the registers
    (1500, 4200, 1, "bf16", True, 1),        # (single values)
]


@pytest.mark.parametrize("shape", GATE, ids=str)
def test_gated_norm_turns(torch_cuda, shape):
    from selective_state_space_63_amd import block
    torch = torch_cuda
    rows, dim, groups, dtype, after, wide = shape
    print(f"[case] gated norm {shape}", flush=True)
    g = np.random.default_rng([52, rows, dim])
    y = put(torch, 2 * g.standard_normal((rows, dim)), dtype, wide)
    z = put(torch, 2 * g.standard_normal((rows, dim)), dtype, 2 * wide)
    w = put(torch, 1 + 0.3 * g.standard_normal(dim), "f32")
    out = block.gated_norm_fwd(y, z, w, groups=groups, gate_after=after, eps=EPS)
    ro = ref.gated_norm(f64(y), f64(z), f64(w), groups, after, EPS)
    close(out, ro, np.abs(ro), "out")
    do = put(torch, g.standard_normal((rows, dim)), dtype)
    got = block.gated_norm_bwd(do, y, z, w, groups=groups, gate_after=after, eps=EPS)
    yv, d, zv = f64(y), f64(do), f64(z)
    sg = 1 / (1 + np.exp(-zv))
    f, df, mdf = zv * sg, sg * (1 + zv * (1 - sg)), sg * (1 + np.abs(zv) * (1 - sg))
    if after:
        du, mdu, dw, mdw = ref.rms_bwd(yv, d * f, f64(w), groups, EPS)
        dz = d * ref.rms(yv, groups, EPS) * f64(w)
        mdz = np.abs(dz)
    else:
        du, mdu, dw, mdw = ref.rms_bwd(yv * f, d, f64(w), groups, EPS)
        dz, mdz = du * yv, mdu * np.abs(yv)
        du, mdu = du * f, mdu * np.abs(f)
    close(got["dy"], du, mdu, "dy")
    close(got["dz"], dz * df, mdz * mdf, "dz")
    close(got["dweight"], dw, mdw, "dweight")
