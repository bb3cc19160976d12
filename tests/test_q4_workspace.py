"""The binding asks for a workspace wherever the library needs one (no GPU needed:
sizes for 256 compute units, those that are taken where no device can be asked)."""
import ctypes

import pytest


def test_rows_without_a_workspace_are_those_of_the_library():
    torch = pytest.importorskip("torch")
    from selective_state_space_63_amd import q4
    lib = q4._load()
    out = ctypes.c_size_t(77)
    assert set(q4.FEW) == {torch.float32, torch.bfloat16, torch.float8_e4m3fn}
    for dt, few in q4.FEW.items():
        sizes = {}
        for rows in range(few + 2):
            for inner, outer in ((128, 16), (8192, 16), (8192, 3305), (2560, 10576), (1 << 20, 128)):
                assert lib.s6_q4_linear_workspace_size(rows, inner, outer, 128, q4._XT[dt], ctypes.byref(out)) == 0
                sizes[rows, inner, outer] = out.value
        assert not any(v for (rows, _, _), v in sizes.items() if rows <= few), dt
        # (one row more takes the other kernel, with slices where there are columns for them)
        assert sizes[few + 1, 8192, 16] > 0, dt
