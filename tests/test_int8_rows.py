"""How many rows moe_grouped_gemm_int8 takes: the kernels count rows and the ends of tiles
of up to 256 rows in 32 bits (fake device addresses, no GPU)."""
import ctypes

import pytest

from test_int8_refusals import SHAPE, WORKSPACE, B, gemm, host_only  # noqa: F401

MOST = 2 ** 31 - 256


@host_only
@pytest.mark.parametrize("rows,code", [(MOST, 0), (MOST + 1, SHAPE), (2 ** 31 - 1, SHAPE), (2 ** 31, SHAPE)])
def test_rows(B, rows, code):  # noqa: F811
    n = ctypes.c_size_t()
    assert B.lib().moe_grouped_gemm_int8_workspace_size(rows, 1, 8, 16, ctypes.byref(n)) == code
    assert gemm(B, rows=rows, E=1, N=8, Kd=16, ws_bytes=1024) == (code or WORKSPACE)
    if code == 0:
        assert n.value >= rows * (16 * 2 + 4)
