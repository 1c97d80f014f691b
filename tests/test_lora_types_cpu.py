"""Half-precision tensors are two bytes wide too, and are not bf16: the adapter calls and the few-token
layer refuse them, and the layer with adapters refuses tensors that do not fit it."""
import os

import pytest
import torch

import mxfp4_expert_gemm_amd as moe

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")

bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
i32 = lambda *s: torch.zeros(s, dtype=torch.int32)


def lora(n_in=256, n_out=64, T=4, **kw):
    return moe.Lora(**{**dict(a=bf(2, 8, n_in), b=bf(2, n_out, 8), scale=torch.ones(2), adapter=i32(T)), **kw})


@pytest.mark.parametrize("name", ["a", "b"])
def test_adapters(name):
    lo = lora()
    with pytest.raises(ValueError, match="bf16"):
        moe._lora(lo._replace(**{name: getattr(lo, name).half()}), 4, 256, 64, torch.device("cpu"))


def test_projection(monkeypatch):
    monkeypatch.setattr(moe, "_same_device", lambda *a: None)
    monkeypatch.setattr(moe, "_p", lambda t: 0)
    for x, W, out in ((bf(4, 256).half(), bf(64, 256), None), (bf(4, 256), bf(64, 256).half(), None),
                      (bf(4, 256), bf(64, 256), bf(4, 64).half())):
        with pytest.raises(ValueError, match="bf16"):
            moe.linear_lora(x, W, lora(), out=out)


def layer_args(**kw):
    a = dict(x=bf(4, 256), router_w=bf(8, 256), latent_down=bf(128, 256), latent_up=bf(256, 128),
             expert_blob=torch.zeros(8 * moe.expert_bytes(128, 128), dtype=torch.uint8), k=2)
    return {**a, **kw}


@pytest.mark.parametrize("name", ["x", "router_w", "latent_down", "latent_up"])
@pytest.mark.parametrize("fn", [moe.layer_decode, moe.layer_forward])
def test_layer(name, fn):
    a = layer_args()
    a[name] = a[name].half()
    with pytest.raises(ValueError, match=f"{name} must be a bf16"):
        fn(**a, d_ffn=128, lora_up=lora(128, 256))


@pytest.mark.parametrize("bad", [dict(latent_up=bf(128, 128)), dict(latent_down=bf(128, 128)), dict(router_w=bf(8, 128)),
                                 dict(expert_blob=torch.zeros(100, dtype=torch.uint8)), dict(out=bf(3, 256)),
                                 dict(bias=torch.zeros(7)), dict(routing=dict(topk_idx=i32(4))),
                                 dict(routing=dict(saliency=torch.zeros(8)))])
def test_layer_with_adapters_refuses_what_does_not_fit(bad):
    with pytest.raises(ValueError, match="must be|must hold|smaller"):
        moe.layer_forward(**layer_args(**bad), d_ffn=128, lora_up=lora(128, 256))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int32, torch.float64])
def test_a_workspace_counts_in_bytes(monkeypatch, dtype):
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0

    real = moe.lib()
    a = layer_args()
    monkeypatch.setattr(moe, "lib", lambda: Lib())
    monkeypatch.setattr(moe, "expert_bytes", real.moe_expert_bytes)
    monkeypatch.setattr(moe, "_p", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(moe, "_stream", lambda s: None)
    monkeypatch.setattr(moe, "_same_device", lambda *t: None)
    ws = torch.empty(800, dtype=dtype)
    for fn in (moe.layer_forward, moe.layer_decode):
        fn(**a, d_ffn=128, lora_up=lora(128, 256), workspace=ws)
    moe.linear_lora(a["x"], bf(64, 256), lora(), workspace=ws)
    assert [args[args.index(ws.data_ptr()) + 1] for _, args in seen] == [800 * ws.element_size()] * 3
