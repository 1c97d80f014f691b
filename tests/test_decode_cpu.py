"""Refusals of the few-token layer: they return before anything touches a device, so this runs
without a GPU."""
import ctypes
import os

import pytest
import torch

import mxfp4_expert_gemm_amd as moe
from test_lora_cpu import FAKE, GB, arg

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")


def ref(a):
    return None if a is None else ctypes.byref(a)


def cfg(T=4, d=256, L=128, F=128, E=8, **kw):
    return moe.make_config(T, d, L, F, E, **kw)


def size(c, k=2, down=None, up=None):
    n = ctypes.c_size_t(0)
    return moe.lib().moe_layer_decode_workspace_size(ctypes.byref(c), k, ref(down), ref(up), ctypes.byref(n)), n.value


def call(c, k=2, down=None, up=None, routing=None, x=FAKE, rw=FAKE + GB, wd=FAKE + 2 * GB, wu=FAKE + 3 * GB,
         blob=FAKE + 4 * GB, bias=None, out=FAKE + 5 * GB, ws=FAKE + 6 * GB, ws_bytes=GB):
    return moe.lib().moe_layer_decode(x, rw, wd, wu, blob, k, ctypes.byref(c), bias, ref(down), ref(up), out,
                                      ref(routing), ws, ws_bytes, None)


def test_sizes():
    st, n = size(cfg())
    assert st == 0 and n > 0
    assert size(cfg(), 2, arg(), arg())[1] > n
    assert size(cfg(T=0))[0] == 0
    assert size(cfg(T=8, E=16), 8)[0] == 0
    assert size(cfg(T=9))[0] == -2
    assert size(cfg(T=8, E=16), 9)[0] == -2      # 72 routed rows
    assert size(cfg(T=1, E=64), 64)[0] == 0
    assert size(cfg(num_shared=1, d_ffn_shared=128))[0] == -2
    assert size(cfg(T=-1))[0] == -1
    assert size(cfg(L=160))[0] == -2
    assert size(cfg(), 0)[0] == -1
    assert size(cfg(), 2, arg(R=4))[0] == -1
    assert size(cfg(), 2, None, arg(R=256))[0] == -2
    assert moe.lib().moe_layer_decode_workspace_size(None, 2, None, None, ctypes.byref(ctypes.c_size_t())) == -1
    assert moe.lib().moe_layer_decode_workspace_size(ctypes.byref(cfg()), 2, None, None, None) == -1


def test_refusals():
    c = cfg()
    assert call(cfg(T=0)) == 0
    assert call(cfg(T=9)) == -2
    assert call(cfg(act=1)) == -2
    assert call(cfg(act=5)) == -1
    for name in ("x", "rw", "wd", "wu", "blob", "out"):
        assert call(c, **{name: None}) == -1, name
        assert call(c, **{name: FAKE + 7 * GB + 8}) == -1, name
    assert call(c, bias=FAKE + 2) == -1
    assert call(c, out=FAKE) == -1                       # out over x
    assert call(c, ws=FAKE) == -1 and call(c, ws=FAKE + 5 * GB) == -1
    assert call(c, ws=FAKE + 6 * GB + 8) == -1
    assert call(c, ws=None) == -3
    assert call(c, ws_bytes=size(c)[1] - 1) == -3
    assert call(c, down=arg(), ws_bytes=size(c)[1]) == -3
    assert call(c, up=arg(a=None)) == -1
    assert call(c, down=arg(adapter=FAKE + 2)) == -1
    assert call(c, routing=moe.RoutingOut(saliency=FAKE + 7 * GB)) == -2


def test_binding_refuses_wrong_shapes():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    c = moe.make_config(4, 256, 128, 128, 8)
    good = dict(x=bf(4, 256), router_w=bf(8, 256), latent_down=bf(128, 256), latent_up=bf(256, 128),
                blob=torch.zeros(8 * moe.expert_bytes(128, 128), dtype=torch.uint8), bias=None, out=None, routing=None)
    chk = lambda **kw: moe._decode_shapes(c, 2, **{**good, **kw})
    chk()
    chk(bias=torch.zeros(8), out=bf(4, 256), routing=dict(topk_idx=i32(4, 2), perm=i32(8), logits=None))
    chk(bias=torch.zeros(4, 8))
    for bad in (dict(x=bf(4, 256).float()), dict(router_w=bf(8, 128)), dict(latent_down=bf(256, 128)),
                dict(latent_up=bf(128, 256)), dict(blob=good["blob"][:-1]), dict(bias=torch.zeros(7)),
                dict(bias=torch.zeros(8).double()), dict(out=bf(3, 256)), dict(out=bf(4, 256).float()),
                dict(routing=dict(topk_idx=i32(7))), dict(routing=dict(topk_idx=i32(8).long())),
                dict(routing=dict(expert_offsets=i32(8))), dict(routing=dict(topk_w=i32(8)))):
        with pytest.raises(ValueError):
            chk(**bad)
