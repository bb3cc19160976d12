"""The C ABI of the projections in few bits without a GPU: libs6.so exports
what include/s6_q4.h declares, and its argument checks (before any HIP call)
return the documented codes.  Every call here fails its checks or has no work
that would be launched."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "s6_q4.h")
LIB = os.path.join(ROOT, "selective_state_space_63_amd", "libs6.so")

OK, NULL, SHAPE, DTYPE, UNSUP, ALIGN = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)
HALF = ctypes.c_void_p((1 << 20) + 2)
EIGHT = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from selective_state_space_63_amd import build
        build.build(LIB)
    from selective_state_space_63_amd import q4
    return q4._load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^int (s6_\w+)\(", text, flags=re.M)))
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert len(names) == 4 and not [n for n in names if n not in exported]
    for n in names:
        assert getattr(lib, n).argtypes is not None, n


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "s6_q4.h"\nint main(void) { return S6_E4M3; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", "-o",
                    str(tmp_path / "t.o"), str(src)], check=True)


def test_linear_checks(lib):
    def f(rows=2, inner=128, outer=8, group=64, xt=1, yt=1, x=P, st=128, xs=None, c=P, s=P, y=P):
        return lib.s6_q4_linear(rows, inner, outer, group, xt, yt, x, st, xs, c, s, y, None, 0, None)

    assert f(xt=3) == DTYPE and f(yt=2) == DTYPE and f(xt=-1) == DTYPE
    assert f(rows=-1) == SHAPE and f(outer=-1) == SHAPE and f(inner=0) == SHAPE and f(st=127) == SHAPE
    assert f(inner=96) == SHAPE and f(inner=96, group=32, st=96, rows=0) == OK
    assert f(group=16) == UNSUP and f(group=256, inner=256, st=256) == UNSUP and f(group=0) == UNSUP
    assert f(outer=1 << 40) == SHAPE and f(rows=1 << 40, st=1 << 40) == SHAPE and f(inner=1 << 30, st=1 << 30) == SHAPE
    assert f(rows=1 << 60, outer=1 << 10) == SHAPE
    assert f(xs=P) == UNSUP and f(xt=2, xs=P, rows=0) == OK and f(outer=0) == OK
    for k in ("x", "c", "s", "y"):
        assert f(**{k: None}) == NULL, k
    assert f(x=ODD) == ALIGN and f(xt=0, x=HALF) == ALIGN and f(c=EIGHT) == ALIGN and f(s=ODD) == ALIGN
    assert f(yt=0, y=HALF) == ALIGN and f(xt=2, xs=HALF) == ALIGN
    out = ctypes.c_size_t(77)
    q = lib.s6_q4_linear_workspace_size
    assert q(2, 128, 8, 64, 1, None) == NULL and q(2, 128, 8, 64, 3, ctypes.byref(out)) == DTYPE
    assert q(2, 128, 8, 48, 1, ctypes.byref(out)) == UNSUP and q(2, 128, 8, 64, 1, ctypes.byref(out)) == OK


def test_pack_checks(lib):
    def f(outer=4, inner=128, group=32, dt=1, w=P, st=128, c=P, s=P):
        return lib.s6_q4_pack(outer, inner, group, dt, w, st, c, s, None)

    assert f(dt=2) == DTYPE and f(group=48) == UNSUP and f(inner=100, st=100) == SHAPE and f(st=64) == SHAPE
    assert f(outer=-1) == SHAPE and f(outer=0) == OK
    assert f(w=None) == NULL and f(c=None) == NULL and f(s=None) == NULL
    assert f(w=ODD) == ALIGN and f(c=EIGHT) == ALIGN and f(s=ODD) == ALIGN


def test_norm_checks(lib):
    def f(rows=4, dim=16, dt=1, rt=0, x=P, st=16, r=P, w=P, g=None, out=P, sc=P, ro=P):
        return lib.s6_add_norm_q8_fwd(rows, dim, dt, rt, x, st, r, w, g, 1.0, 1e-5, out, sc, ro, None)

    assert f(dt=2) == DTYPE and f(rt=2) == DTYPE and f(dt=0, rt=1) == DTYPE
    assert f(rows=-1) == SHAPE and f(dim=0) == SHAPE and f(st=15) == SHAPE and f(rows=1 << 40, dim=1 << 30) == SHAPE
    for k in ("x", "w", "out", "sc", "ro"):
        assert f(**{k: None}) == NULL, k
    assert f(x=ODD) == ALIGN and f(r=HALF) == ALIGN and f(g=HALF) == ALIGN and f(sc=HALF) == ALIGN
    assert f(rows=0) == OK


def test_binding_refuses(lib):
    """Shapes, types, layouts and devices that the entry points do not take."""
    torch = pytest.importorskip("torch")
    from selective_state_space_63_amd import q4
    x, w, s = torch.zeros(3, 128), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        q4.q4_linear(x, w, s)
    with pytest.raises(ValueError, match="dtype"):
        q4.q4_linear(x.half(), w, s)
    with pytest.raises(ValueError, match="out_dtype"):
        q4.q4_linear(x, w, s, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="groups"):
        q4.q4_linear(x, w, s[:, :0])
    with pytest.raises(ValueError, match="groups"):
        q4.q4_linear(x[:, :96], w, torch.zeros(8, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="groups"):
        q4.q4_pack(x, 48)
    with pytest.raises(ValueError, match="outer"):
        q4.q4_pack(x[0], 32)
    with pytest.raises(ValueError, match="device"):
        q4.q4_pack(x, 32)
    with pytest.raises(ValueError, match="device"):
        q4.add_norm_q8_fwd(x, torch.ones(128))
