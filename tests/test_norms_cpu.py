"""Refusals of the calls between two blocks: every bad argument returns before anything touches a
device, so this runs without a GPU; and the tests' fp64 gradients agree with differences."""
import ctypes
import os

import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain_norms

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")

FAKE = 0x7F0000000000  # 16-byte aligned; never dereferenced on these paths
GB = 1 << 30


def at(i):
    return FAKE + i * GB


def size(T=8, d=64):
    n = ctypes.c_size_t(0)
    return moe.lib().moe_block_norms_backward_workspace_size(T, d, ctypes.byref(n)), n.value


def forward(T=8, d=64, scale=1.0, eps=1e-6, stride=0, **kw):
    p = dict(y=at(0), r=at(1), post=at(2), pre=at(3), gate=at(4), out=at(5), normed=at(6))
    p.update(kw)
    return moe.lib().moe_block_norms(p["y"], p["r"], p["post"], p["pre"], p["gate"], stride, T, d, scale, eps, p["out"],
                                     p["normed"], None)


def backward(T=8, d=64, scale=1.0, eps=1e-6, stride=0, **kw):
    p = dict(dout=at(0), dn=at(1), y=at(2), out=at(3), post=at(4), pre=at(5), gate=at(6), dr=at(7), dy=at(8), dpost=at(9),
             dpre=at(10), dgate=at(11), ws=at(12), ws_bytes=GB)
    p.update(kw)
    return moe.lib().moe_block_norms_backward(p["dout"], p["dn"], p["y"], p["out"], p["post"], p["pre"], p["gate"], stride, T,
                                              d, scale, eps, p["dr"], p["dy"], p["dpost"], p["dpre"], p["dgate"], p["ws"],
                                              p["ws_bytes"], None)


def test_workspace_size():
    assert size()[0] == 0 and size()[1] >= 3 * 64 * 4
    assert size(T=0) == (0, 0)
    for bad in (dict(T=-1), dict(d=0), dict(d=60)):
        assert size(**bad)[0] == -1
    assert size(d=8200)[0] == -2 and size(T=(1 << 24) + 1)[0] == -2
    assert moe.lib().moe_block_norms_backward_workspace_size(8, 64, None) == -1


def test_forward_refusals():
    nan, inf = float("nan"), float("inf")
    assert forward(T=0) == 0
    for bad in (dict(r=None), dict(out=None), dict(normed=None), dict(pre=None), dict(y=None), dict(y=None, out=None),
                dict(y=None, out=None, post=None, gate=None, pre=None, normed=None), dict(y=at(0) + 8), dict(pre=at(3) + 2),
                dict(gate=at(4) + 4), dict(out=at(5) + 8), dict(normed=at(6) + 1), dict(out=at(0)), dict(normed=at(5)),
                dict(normed=at(1)), dict(out=at(1) + 16), dict(out=at(2)), dict(d=60), dict(d=0), dict(T=-1), dict(stride=32),
                dict(scale=nan), dict(scale=inf), dict(eps=-1e-6), dict(eps=nan), dict(eps=inf)):
        assert forward(**bad) == -1, bad
    assert forward(d=8200) == -2 and forward(T=(1 << 24) + 1) == -2


def test_backward_refusals():
    assert backward(T=0, dpost=None, dpre=None, dgate=None) == 0
    for bad in (dict(dout=None, dn=None), dict(out=None), dict(pre=None, dpre=None), dict(pre=None, dpre=None, out=None),
                dict(y=None), dict(post=None), dict(gate=None), dict(dout=at(0) + 8), dict(dr=at(1)), dict(dr=at(0) + 16),
                dict(dy=at(2)), dict(dy=at(7)), dict(dpost=at(9) + 4), dict(dpre=at(9)), dict(dgate=at(3)), dict(ws=at(11)),
                dict(ws=at(12) + 8), dict(d=60), dict(stride=8), dict(eps=-1.0)):
        assert backward(**bad) == -1, bad
    assert backward(ws=None) == -3 and backward(ws_bytes=size()[1] - 1) == -3
    assert backward(d=8200) == -2


def test_binding_refusals():
    def b(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype)

    ok = dict(y=b(4, 64), residual=b(4, 64), pre_weight=b(64), post_weight=b(64), gate=b(64))
    for bad in (dict(y=b(4, 56)), dict(residual=b(3, 64)), dict(pre_weight=b(4, 64)), dict(post_weight=b(64, dtype=torch.float32)),
                dict(gate=b(4)), dict(gate=b(4, 1)), dict(out=b(4, 56)), dict(normed=b(64, 4)), dict(y=None),
                dict(pre_weight=None, normed=b(4, 64)), dict(residual=b(4, 64, dtype=torch.float16))):
        with pytest.raises(ValueError):
            moe.block_norms(**{**ok, **bad})
    back = dict(dout=b(4, 64), dnormed=b(4, 64), y=b(4, 64), out=b(4, 64), pre_weight=b(64), post_weight=b(64), gate=b(64))
    none = moe.BlockNormsGrads(None, None, None, None, None)
    for bad in (dict(dout=None, dnormed=None), dict(out=None), dict(pre_weight=None), dict(y=None), dict(gate=b(8)),
                dict(grads=none._replace(dy=b(4, 64, dtype=torch.float32))), dict(grads=none._replace(dgate=b(64))),
                dict(grads=none._replace(dpre_weight=b(64))), dict(dnormed=b(4, 72))):
        with pytest.raises(ValueError):
            moe.block_norms_backward(**{**back, **bad})


def test_plain_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    at_ = dict(y=n(4, 16), residual=n(4, 16), post=n(16), pre=n(16), gate=n(4, 16))
    dout, dn, eps = n(4, 16), n(4, 16), 1e-3

    def outputs(v):
        out = v["residual"] + 0.5 * v["gate"] * plain_norms.norm(v["y"], eps)[0] * v["post"]
        return out, plain_norms.norm(out, eps)[0] * v["pre"]

    out = outputs(at_)[0]
    want = plain_norms.backward(dout, dn, at_["y"], out, at_["pre"], at_["post"], at_["gate"], 0.5, eps)
    for grad, name in dict(dy="y", dresidual="residual", dpost_weight="post", dpre_weight="pre", dgate="gate").items():
        v = n(*at_[name].shape)
        f = lambda s: sum((a * b).sum() for a, b in zip(outputs({**at_, name: at_[name] + s * v}), (dout, dn)))
        slope = (f(1e-6) - f(-1e-6)) / 2e-6
        assert abs(slope - (want[grad][0] * v).sum()) <= 1e-6 * (1 + abs(slope)), name
