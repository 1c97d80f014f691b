"""Refusals of the 8-bit calls: every bad argument returns before anything touches a device, so this
runs without a GPU; and the tests' plain quantiser on values done by hand."""
import ctypes
import os

import numpy as np
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
from plain_int8 import codes

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")

FAKE = 0x7F0000000000  # 16-byte aligned; never dereferenced on these paths
GB = 1 << 30


def at(i):
    return FAKE + i * GB


def size(T=8, n_in=64, n_out=33, quantize=1):
    n = ctypes.c_size_t(0)
    return moe.lib().moe_linear_int8_workspace_size(T, n_in, n_out, quantize, ctypes.byref(n)), n.value


def linear(T=8, n_in=64, n_out=33, **kw):
    p = dict(x=at(0), xs=None, W=at(2), ws=at(3), out=at(4), work=at(5), work_bytes=GB)
    p.update(kw)
    return moe.lib().moe_linear_int8(p["x"], p["xs"], p["W"], p["ws"], T, n_in, n_out, p["out"], p["work"], p["work_bytes"],
                                     None)


def quantize(rows=8, n=64, x=at(0), q=at(1), scale=at(2)):
    return moe.lib().moe_quantize_int8(x, rows, n, q, scale, None)


def test_workspace_size():
    assert size()[0] == 0 and size()[1] >= 8 * 64 + 8 * 4
    assert size(T=0) == (0, 0) and size(quantize=0) == (0, 0)
    for bad in (dict(T=-1), dict(n_in=0), dict(n_in=24), dict(n_out=0)):
        assert size(**bad)[0] == -1
    assert size(n_in=65552)[0] == -2 and size(T=(1 << 24) + 1)[0] == -2
    assert moe.lib().moe_linear_int8_workspace_size(8, 64, 33, 1, None) == -1


def test_call_refusals():
    assert linear(T=0) == 0
    for bad in (dict(x=None), dict(W=None), dict(ws=None), dict(out=None), dict(x=at(0) + 8), dict(W=at(2) + 8),
                dict(ws=at(3) + 4), dict(xs=at(1) + 4), dict(out=at(4) + 2), dict(out=at(0)), dict(out=at(2)),
                dict(work=at(4)), dict(work=at(0)), dict(work=at(5) + 8), dict(n_in=24), dict(n_out=0), dict(T=-1)):
        assert linear(**bad) == -1, bad
    assert linear(work=None) == -3 and linear(work_bytes=size()[1] - 1) == -3
    assert linear(n_in=65552) == -2
    assert quantize(rows=0) == 0
    for bad in (dict(x=None), dict(q=None), dict(scale=None), dict(x=at(0) + 8), dict(q=at(1) + 4), dict(scale=at(2) + 4),
                dict(q=at(0)), dict(scale=at(1)), dict(n=8), dict(rows=-1)):
        assert quantize(**bad) == -1, bad
    assert quantize(n=65552) == -2


def test_binding_refusals():
    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype)

    i8, f32 = torch.int8, torch.float32
    ok = dict(inp=t(4, 64), W=t(40, 64, dtype=i8), w_scale=t(40, dtype=f32))
    for bad in (dict(inp=t(4, 48)), dict(inp=t(4, 64, dtype=f32)), dict(inp=t(4, 64, dtype=i8)), dict(W=t(40, 64)),
                dict(w_scale=t(40)), dict(w_scale=t(64, dtype=f32)), dict(x_scale=t(4, dtype=f32)),
                dict(inp=t(4, 64, dtype=i8), x_scale=t(5, dtype=f32)), dict(out=t(4, 64))):
        with pytest.raises(ValueError):
            moe.linear_int8(**{**ok, **bad})
    for bad in (dict(x=t(4, 64, dtype=f32)), dict(x=t(4, 64), q=t(4, 64)), dict(x=t(4, 64), scale=t(4))):
        with pytest.raises(ValueError):
            moe.quantize_int8(**bad)


def test_plain_codes_by_hand():
    x = torch.tensor([[2.0, 1.0, -1.0, 0.0], [254.0, 1.0, 3.0, -5.0], [0.0, 0.0, 0.0, 0.0]], dtype=torch.bfloat16)
    q, s = codes(x)
    # 127 / 2 = 63.5 -> 64; 0.5 -> 0, 1.5 -> 2, -2.5 -> -2
    assert q.tolist() == [[127, 64, -64, 0], [127, 0, 2, -2], [0, 0, 0, 0]]
    assert s.tolist() == [np.float32(2) / np.float32(127), 2.0, 0.0]
