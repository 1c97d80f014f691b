"""linear_int8 refuses more columns than its tiles number in 32 bits, before anything touches a device."""
import ctypes
import os

import pytest

import mxfp4_expert_gemm_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")


@pytest.mark.parametrize("n_out,status", [(2 ** 31 - 256, 0), (2 ** 31 - 255, -2), (2 ** 31 - 1, -2)])
def test_columns(n_out, status):
    n = ctypes.c_size_t(0)
    assert moe.lib().moe_linear_int8_workspace_size(1, 16, n_out, 0, ctypes.byref(n)) == status
    if status:  # the addresses are never used
        p = [0x7F0000000000 + (i << 40) for i in range(4)]
        assert moe.lib().moe_linear_int8(p[0], p[1], p[2], p[3], 1, 16, n_out, p[0] + (1 << 43), None, 0, None) == status
