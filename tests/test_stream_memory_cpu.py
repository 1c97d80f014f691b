"""What a call allocates for itself comes from the memory of the stream it runs on.  The library and
the CUDA streams are stand-ins, so this runs without a GPU: a buffer of another stream's memory
is never handed to a kernel."""
import contextlib

import pytest
import torch

import mxfp4_expert_gemm_amd as moe

bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
T, D, L, F, E, K = 4, 256, 128, 128, 8, 2


class Stream:
    cuda_stream = 5


class Pinned(torch.Tensor):
    def is_pinned(self, *a):
        return True


@pytest.fixture
def seen(monkeypatch):
    """Per allocation, the stream whose memory it is (None: the current one's)."""
    on, got, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    def alloc(*a, **kw):
        got.append(on[-1])
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p: p)  # the stand-in's stream by its pointer
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch, "empty", alloc)
    monkeypatch.setattr(moe, "lib", lambda: Lib())
    monkeypatch.setattr(moe, "_p", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(moe, "_same_device", lambda *a: None)
    monkeypatch.setattr(moe, "expert_bytes", lambda *a: 16)
    return got


def lora(n_in, n_out):
    return moe.Lora(bf(2, 8, n_in), bf(2, n_out, 8), torch.ones(2), torch.zeros(T, dtype=torch.int32))


LAYER = (bf(T, D), bf(E, D), bf(L, D), bf(D, L), torch.zeros(E * 16, dtype=torch.uint8), K)
ADAPTERS = dict(lora_down=lora(D, L), lora_up=lora(L, D))
HOST = LAYER[:4] + (LAYER[4].as_subclass(Pinned), K)
CALLS = {
    "linear_lora": (lambda **kw: moe.linear_lora(bf(T, D), bf(L, D), lora(D, L), **kw), 2),
    "layer_decode": (lambda **kw: moe.layer_decode(*LAYER, d_ffn=F, **kw), 2),
    "layer_decode_lora": (lambda **kw: moe.layer_decode(*LAYER, d_ffn=F, **ADAPTERS, **kw), 2),
    "layer_forward": (lambda **kw: moe.layer_forward(*LAYER, d_ffn=F, **kw), 2),
    "layer_forward_lora": (lambda **kw: moe.layer_forward(*LAYER, d_ffn=F, **ADAPTERS, **kw), 2),
    "layer_forward_profiled": (lambda **kw: moe.layer_forward_profiled(*LAYER, moe.StageEvents(), d_ffn=F, **kw), 2),
    "layer_forward_streamed": (lambda **kw: moe.layer_forward_streamed(*HOST, d_ffn=F, **kw), 3),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_belong_to_the_stream_of_the_call(seen, name):
    call, n = CALLS[name]
    s = Stream()
    call(stream=s)
    assert seen == [s.cuda_stream] * n
    seen.clear()
    call()
    assert seen == [None] * n
