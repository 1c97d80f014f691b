"""LayerStack.forward refuses what does not fit before any layer has run, the last argument and the last
layer's among it."""
import os

import pytest
import torch

import mxfp4_expert_gemm_amd as moe
from mxfp4_expert_gemm_amd import stream

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="libmoe_layer.so not built")

T, D, F, E, L = 4, 64, 72, 8, 128


class Ran(Exception):
    pass


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def dense(**kw):
    return dict(w_gate=bf16(F, D), w_up=bf16(F, D), w_down=bf16(D, F), **kw)


def routed(monkeypatch, **kw):
    monkeypatch.setattr(torch.Tensor, "is_pinned", lambda self: True)
    monkeypatch.setattr(stream, "alloc_workspace", lambda *a: None)
    monkeypatch.setattr(stream, "alloc_expert_slots", lambda *a: None)
    lay = dict(router_w=bf16(E, D), latent_down=bf16(L, D), latent_up=bf16(D, L),
               expert_blob_host=torch.zeros(E * moe.expert_bytes(L, 128), dtype=torch.uint8))
    lay.update(kw)
    return lay


def run(monkeypatch, layers, x=None, **kw):
    """The stack's forward with calls that only say that they were reached."""
    def ran(*a, **k):
        raise Ran

    s = stream.LayerStack(layers, 2, 128, 0, T, device="cpu")
    for name in ("block_norms", "gated_ffn", "layer_forward", "layer_forward_streamed"):
        monkeypatch.setattr(stream, name, ran)
    return s.forward(bf16(T, D) if x is None else x, **kw)


def int8_head(n=32, d=D):
    return torch.zeros(n, d, dtype=torch.int8), torch.ones(n)


def test_what_fits_runs(monkeypatch):
    full = dict(pre_norm=bf16(D), post_norm=bf16(D), gate=bf16(T, D), scale=0.5)
    for kw in (dict(), dict(final_norm=bf16(D)), dict(final_norm=bf16(D), head=int8_head()),
               dict(final_norm=bf16(D), head=bf16(32, D)), dict(eps=0.0)):
        with pytest.raises(Ran):
            run(monkeypatch, [dense(**full), dense(gate=bf16(D))], **kw)
    for bias in (None, torch.zeros(E), torch.zeros(T, E)):
        with pytest.raises(Ran):
            run(monkeypatch, [routed(monkeypatch, bias=bias, **full)])
    x = bf16(T, D)
    assert run(monkeypatch, [], x=x) == (x, None)


@pytest.mark.parametrize("name,kw", [
    ("codes too narrow", dict(final_norm=bf16(D), head=int8_head(d=D - 16))),
    ("codes in bf16", dict(final_norm=bf16(D), head=(bf16(32, D), torch.ones(32)))),
    ("scales in fp64", dict(final_norm=bf16(D), head=(int8_head()[0], torch.ones(32, dtype=torch.float64)))),
    ("one scale short", dict(final_norm=bf16(D), head=(int8_head()[0], torch.ones(31)))),
    ("codes transposed", dict(final_norm=bf16(D), head=(torch.zeros(D, 32, dtype=torch.int8).t(), torch.ones(32)))),
    ("a head without a norm", dict(head=int8_head())),
    ("a bf16 head too narrow", dict(final_norm=bf16(D), head=bf16(32, D - 8))),
    ("final_norm too long", dict(final_norm=bf16(D + 8))),
    ("final_norm in fp32", dict(final_norm=torch.zeros(D))),
    ("every second of final_norm", dict(final_norm=bf16(2 * D)[::2])),
    ("eps below zero", dict(eps=-1e-6)),
    ("eps not a number", dict(eps=float("nan"))),
    ("eps past fp32", dict(eps=1e39)),
])
def test_arguments(monkeypatch, name, kw):
    with pytest.raises(ValueError):
        run(monkeypatch, [dense()], **kw)


@pytest.mark.parametrize("name,kw", [
    ("pre_norm", dict(pre_norm=bf16(D - 8))), ("pre_norm", dict(pre_norm=torch.zeros(D))),
    ("post_norm", dict(post_norm=bf16(1, D))), ("post_norm", dict(post_norm=bf16(2 * D)[::2])),
    ("gate", dict(gate=bf16(T + 1, D))), ("gate", dict(gate=torch.zeros(D))), ("gate", dict(gate=bf16(D, T).t())),
    ("scale", dict(scale=float("inf"))), ("scale", dict(scale=float("nan"))), ("scale", dict(scale=-1e39)),
    ("w_up", dict(w_up=bf16(F + 8, D))), ("w_down", dict(w_down=bf16(F, D))), ("w_down", dict(w_down=bf16(F, D).t())),
])
def test_the_last_dense_layer(monkeypatch, name, kw):
    with pytest.raises(ValueError):
        run(monkeypatch, [dense(), {**dense(), **kw}])


@pytest.mark.parametrize("name,kw", [
    ("latent_up", dict(latent_up=bf16(L, D))), ("router_w", dict(router_w=torch.zeros(E, D))),
    ("latent_down", dict(latent_down=bf16(D, L).t())), ("bias", dict(bias=torch.zeros(E + 1))),
    ("bias", dict(bias=torch.zeros(E, dtype=torch.float64))), ("bias", dict(bias=torch.zeros(T + 1, E))),
    ("experts", dict(expert_blob_host=torch.zeros(E * moe.expert_bytes(L, 128) - 1, dtype=torch.uint8))),
    ("post_norm", dict(post_norm=bf16(D + 8))),
])
def test_the_last_routed_layer(monkeypatch, name, kw):
    with pytest.raises(ValueError):
        run(monkeypatch, [dense(), routed(monkeypatch, **kw)])


def test_width_of_an_8_bit_head(monkeypatch):
    d = 72  # a width for every other call
    lay = dict(w_gate=bf16(F, d), w_up=bf16(F, d), w_down=bf16(d, F))
    with pytest.raises(ValueError):
        run(monkeypatch, [lay], x=bf16(T, d), final_norm=bf16(d), head=int8_head(d=d))
