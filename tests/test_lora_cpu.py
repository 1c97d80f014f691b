"""Refusals of the adapter calls: every bad argument returns before anything touches a device,
so this runs without a GPU; and the tests' plain forms hold on cases done by hand."""
import ctypes
import os

import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")

FAKE = 0x7F0000000000  # 16-byte aligned; never dereferenced on these paths
GB = 1 << 30


def arg(N=4, R=16, **kw):
    p = dict(a=FAKE + 10 * GB, b=FAKE + 11 * GB, scale=FAKE + 12 * GB, rank=None, adapter=FAKE + 13 * GB)
    p.update(kw)
    return moe.LoraArg(p["a"], p["b"], p["scale"], p["rank"], p["adapter"], N, R)


def size(T=8, n_in=256, lo=None):
    n = ctypes.c_size_t(0)
    lo = lo if lo is not None else arg()
    return moe.lib().moe_linear_lora_workspace_size(T, n_in, ctypes.byref(lo), ctypes.byref(n)), n.value


def call(T=8, n_in=256, n_out=128, lo=None, x=FAKE, W=FAKE + GB, out=FAKE + 2 * GB, ws=FAKE + 3 * GB, ws_bytes=GB):
    lo = lo if lo is not None else arg()
    return moe.lib().moe_linear_lora(x, W, ctypes.byref(lo), T, n_in, n_out, out, ws, ws_bytes, None)


def test_workspace_size():
    st, n = size()
    assert st == 0 and n >= 8 * 16 * 4
    assert size(T=0) == (0, 0)
    assert size(T=4096)[1] > size(T=64)[1]
    assert size(lo=arg(a=None, b=None, scale=None, adapter=None))[0] == 0  # sizes only
    assert size(T=-1)[0] == -1
    assert size(n_in=100)[0] == -1
    assert size(n_in=8224)[0] == -2
    assert size(T=(1 << 24) + 1)[0] == -2
    assert size(lo=arg(N=0))[0] == -1
    assert size(lo=arg(N=1025))[0] == -2
    assert size(lo=arg(R=12))[0] == -1
    assert size(lo=arg(R=0))[0] == -1
    assert size(lo=arg(R=136))[0] == -2
    lib = moe.lib()
    assert lib.moe_linear_lora_workspace_size(1, 256, None, ctypes.byref(ctypes.c_size_t())) == -1
    assert lib.moe_linear_lora_workspace_size(1, 256, ctypes.byref(arg()), None) == -1


def test_call_refusals():
    assert call(T=0) == 0
    assert call(T=0, x=None, W=None, out=None, ws=None) == 0
    for bad in (dict(x=None), dict(W=None), dict(out=None), dict(x=FAKE + 8), dict(W=FAKE + GB + 8),
                dict(out=FAKE + 2 * GB + 1), dict(n_out=0), dict(T=-1), dict(n_in=100), dict(ws=FAKE + 3 * GB + 4),
                dict(out=FAKE + 16), dict(ws=FAKE), dict(ws=FAKE + 2 * GB), dict(lo=arg(a=None)),
                dict(lo=arg(b=None)), dict(lo=arg(scale=None)), dict(lo=arg(adapter=None)),
                dict(lo=arg(a=FAKE + 8)), dict(lo=arg(b=FAKE + 8)), dict(lo=arg(scale=FAKE + 2)),
                dict(lo=arg(adapter=FAKE + 2)), dict(lo=arg(rank=FAKE + 2)), dict(lo=arg(R=4))):
        assert call(**bad) == -1, bad
    assert moe.lib().moe_linear_lora(FAKE, FAKE, None, 1, 256, 128, FAKE, FAKE, GB, None) == -1
    assert call(ws=None) == -3
    assert call(ws_bytes=size()[1] - 1) == -3
    assert call(lo=arg(R=256)) == -2


def layer(cfg, down=None, up=None, k=2, ws_bytes=1 << 40):
    ref = lambda a: None if a is None else ctypes.byref(a)
    return moe.lib().moe_layer_forward_lora(FAKE, FAKE + GB, FAKE + 2 * GB, FAKE + 3 * GB, FAKE + 4 * GB, k,
                                            ctypes.byref(cfg), None, None, ref(down), ref(up), FAKE + 5 * GB, None,
                                            FAKE + (1 << 41), ws_bytes, None)


def layer_size(cfg, k, down, up):
    n = ctypes.c_size_t(0)
    ref = lambda a: None if a is None else ctypes.byref(a)
    return moe.lib().moe_layer_lora_workspace_size(ctypes.byref(cfg), k, ref(down), ref(up), ctypes.byref(n)), n.value


def test_layer_refusals():
    cfg = moe.make_config(8, 256, 128, 128, 8)
    base = moe.workspace_size(cfg, 2)
    assert layer_size(cfg, 2, None, None) == (0, base)
    st, need = layer_size(cfg, 2, arg(), arg(R=64))
    assert st == 0 and need > base
    assert layer(cfg, arg(), arg(R=64), ws_bytes=need - 1) == -3
    assert layer(cfg, arg(a=None)) == -1
    assert layer(cfg, None, arg(scale=FAKE + 1)) == -1
    assert layer(cfg, arg(N=0)) == -1
    assert layer(cfg, None, arg(R=200)) == -2
    assert layer(moe.make_config(0, 256, 128, 128, 8), arg(), arg()) == 0
    assert layer_size(cfg, 0, None, None)[0] == -1


def test_binding_refuses_wrong_shapes():
    x, W = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros((64, 256), dtype=torch.bfloat16)
    lo = dict(a=torch.zeros((2, 8, 256), dtype=torch.bfloat16), b=torch.zeros((2, 64, 8), dtype=torch.bfloat16),
              scale=torch.ones(2), adapter=torch.zeros(4, dtype=torch.int32))
    chk = lambda **kw: moe._lora(moe.Lora(**{**lo, **kw}), 4, 256, 64, torch.device("cpu"))
    for bad in (dict(a=lo["a"][:, :, :128]), dict(a=lo["a"].float()), dict(b=lo["b"][:, :32]), dict(b=lo["b"].float()),
                dict(scale=torch.ones(3)), dict(scale=torch.ones(2).double()), dict(adapter=lo["adapter"][:3]),
                dict(adapter=lo["adapter"].long()), dict(rank=torch.ones(1, dtype=torch.int32)),
                dict(rank=torch.ones(2)), {}):  # the last: not on a GPU
        with pytest.raises(ValueError):
            chk(**bad)


def test_plain_forms_by_hand():
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]).bfloat16()
    W = torch.tensor([[1.0, 0.0], [0.0, 2.0]]).bfloat16()
    lo = dict(a=torch.tensor([[[1.0, 1.0], [0.0, 1.0]]]).bfloat16(), b=torch.tensor([[[1.0, 10.0], [0.0, 1.0]]]).bfloat16(),
              scale=torch.tensor([0.5]))
    v, _ = plain.linear(x, W, lo, torch.tensor([0, -1, 0]))
    # token 0: u = (3, 2), b u = (23, 2); token 2: u = (11, 6), b u = (71, 6)
    assert torch.equal(v, torch.tensor([[1 + 11.5, 4 + 1.0], [3.0, 8.0], [5 + 35.5, 12 + 3.0]]).double())
    v, _ = plain.linear(x, W, lo, torch.tensor([0, -1, 1]), torch.tensor([1]))
    assert torch.equal(v, torch.tensor([[1 + 1.5, 4.0], [3.0, 8.0], [5.0, 12.0]]).double())
    q = plain.mxfp8(torch.tensor([[300.0, 0.3, -17.0, 1e-5] + [0.0] * 28]).double())[0]
    # top 300: scale 2^0, steps of 32 at 300, of 1/32 at 0.3, of 2 at 17 (a tie, to the even 16)
    assert q[:4].tolist() == [288.0, 0.3125, -16.0, 0.0]
