"""Refusals of the dense block's calls: every bad argument returns before anything touches a device,
so this runs without a GPU; and the tests' fp64 gradients agree with differences."""
import ctypes
import os

import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain_ffn

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")

FAKE = 0x7F0000000000  # 16-byte aligned; never dereferenced on these paths
GB = 1 << 30


def at(i):
    return FAKE + i * GB


def size(T=8, d=64, F=72, backward=False):
    n = ctypes.c_size_t(0)
    f = moe.lib().moe_gated_ffn_backward_workspace_size if backward else moe.lib().moe_gated_ffn_workspace_size
    return f(T, d, F, ctypes.byref(n)), n.value


def forward(T=8, d=64, F=72, **kw):
    p = dict(x=at(0), wg=at(1), wu=at(2), wd=at(3), out=at(4), gate=None, up=None, ws=at(7), ws_bytes=GB)
    p.update(kw)
    return moe.lib().moe_gated_ffn(p["x"], p["wg"], p["wu"], p["wd"], T, d, F, p["out"], p["gate"], p["up"], p["ws"],
                                   p["ws_bytes"], None)


def backward(T=8, d=64, F=72, **kw):
    p = dict(dout=at(0), x=at(1), wg=at(2), wu=at(3), wd=at(4), gate=at(5), up=at(6), dx=at(7), dwg=at(8), dwu=at(9),
             dwd=at(10), ws=at(11), ws_bytes=GB)
    p.update(kw)
    return moe.lib().moe_gated_ffn_backward(p["dout"], p["x"], p["wg"], p["wu"], p["wd"], p["gate"], p["up"], T, d, F,
                                            p["dx"], p["dwg"], p["dwu"], p["dwd"], p["ws"], p["ws_bytes"], None)


@pytest.mark.parametrize("back", [False, True])
def test_workspace_size(back):
    assert size(backward=back)[0] == 0 and size(backward=back)[1] >= 8 * 72 * 2
    assert size(T=0, backward=back) == (0, 0)
    for bad in (dict(T=-1), dict(d=0), dict(F=0), dict(d=60), dict(F=4)):
        assert size(**bad, backward=back)[0] == -1, bad
    for big in (dict(T=(1 << 24) + 1), dict(d=32776), dict(F=32776)):
        assert size(**big, backward=back)[0] == -2, big
    f = moe.lib().moe_gated_ffn_backward_workspace_size if back else moe.lib().moe_gated_ffn_workspace_size
    assert f(8, 64, 72, None) == -1


def test_forward_refusals():
    assert forward(T=0) == 0 and forward(T=0, x=None, wg=None, out=None, ws=None) == 0
    for bad in (dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(out=None), dict(x=FAKE + 8),
                dict(wg=at(1) + 2), dict(out=at(4) + 8), dict(gate=at(5)), dict(up=at(6)), dict(gate=at(5) + 4, up=at(6)),
                dict(gate=at(5), up=at(5)), dict(out=FAKE), dict(out=at(3)), dict(ws=at(4)), dict(ws=at(7) + 4),
                dict(gate=at(5), up=at(4)), dict(d=60), dict(T=-1)):
        assert forward(**bad) == -1, bad
    assert forward(ws=None) == -3 and forward(ws_bytes=size()[1] - 1) == -3
    assert forward(F=40000) == -2


def test_backward_refusals():
    assert backward(T=0, dx=at(7), dwg=None, dwu=None, dwd=None) == 0
    for name in ("dout", "x", "wg", "wu", "wd", "gate", "up"):
        assert backward(**{name: None}) == -1, name
        assert backward(**{name: at(20) + 8}) == -1, name
    for bad in (dict(dwg=None), dict(dwu=None), dict(dwd=None), dict(dx=None, dwg=None, dwu=None, dwd=None),
                dict(dx=at(0)), dict(dx=at(1)), dict(dwg=at(2)), dict(dwg=at(9)), dict(dwd=at(4)), dict(dx=at(7) + 8),
                dict(ws=at(6)), dict(ws=at(10)), dict(dwg=at(8) + 2), dict(F=36)):
        assert backward(**bad) == -1, bad
    assert backward(ws=None) == -3 and backward(ws_bytes=size(backward=True)[1] - 1) == -3
    assert backward(dwg=None, dwu=None, dwd=None, ws=None) == -3
    assert backward(d=40000) == -2


def test_binding_refusals():
    def b(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype)

    ok = dict(x=b(4, 64), w_gate=b(72, 64), w_up=b(72, 64), w_down=b(64, 72))
    for bad in (dict(x=b(4, 56)), dict(w_up=b(64, 72)), dict(w_down=b(72, 64)), dict(x=b(4, 64, dtype=torch.float16)),
                dict(w_gate=b(72, 64, dtype=torch.float32)), dict(out=b(4, 72)), dict(gate=b(4, 72)),
                dict(gate=b(4, 64), up=b(4, 72))):
        with pytest.raises(ValueError):
            moe.gated_ffn(**{**ok, **bad})
    back = dict(dout=b(4, 64), **ok, gate=b(4, 72), up=b(4, 72))
    none = moe.GatedFfnGrads(None, None, None, None)
    for bad in (dict(dout=b(3, 64)), dict(gate=b(4, 64)), dict(up=b(4, 72, dtype=torch.float32)),
                dict(want_dx=False, want_dw=False), dict(want_dx=False, out=none._replace(dx=b(4, 64))),
                dict(out=none._replace(dw_up=b(64, 72)))):
        with pytest.raises(ValueError):
            moe.gated_ffn_backward(**{**back, **bad})


def test_plain_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    x, wg, wu, wd, dout = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((5, 8), (16, 8), (16, 8), (8, 16), (5, 8)))

    def loss(x, wg, wu, wd):
        return (plain_ffn.forward(x, wg, wu, wd)["out"][0] * dout).sum()

    kept = plain_ffn.forward(x, wg, wu, wd)
    want = plain_ffn.backward(dout, x, wg, wu, wd, kept["gate"][0], kept["up"][0])
    args = [x, wg, wu, wd]
    for i, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-6 * v, args[i] - 1e-6 * v
        slope = (loss(*up) - loss(*down)) / 2e-6
        assert abs(slope - (want[name][0] * v).sum()) <= 1e-6 * (1 + abs(slope))
