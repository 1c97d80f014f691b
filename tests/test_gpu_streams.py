"""Calls on a side stream that allocate for themselves: their buffers stay theirs while the current
stream goes on allocating and writing."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
from test_gpu_decode import Layer
from test_gpu_lora import dev_lora, ids_of

pytestmark = pytest.mark.gpu


def beside(call, want):
    """The call on a side stream behind some milliseconds of other work, while the current stream
    writes over all memory that is free to it."""
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(10_000_000)
        out = call(side)
        trash = [torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (64, 4096, 1 << 16, 1 << 20, 1 << 22) * 4]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        out.record_stream(torch.cuda.current_stream())
        del out, trash


@pytest.mark.parametrize("T,R", [(3, 16), (40, 16), (700, 32)])
def test_linear_lora(T, R):
    lo = plain.adapters(4, R, 512, 320, 3)
    x, W = plain.bf16((T, 512), 1.0, 1).cuda(), plain.bf16((320, 512), 0.05, 2).cuda()
    l = dev_lora(lo, ids_of(T, 4, "mixed", 1))
    beside(lambda s: moe.linear_lora(x, W, l, stream=s), moe.linear_lora(x, W, l))


@pytest.mark.parametrize("T,fn", [(3, moe.layer_decode), (3, moe.layer_forward), (40, moe.layer_forward)])
@pytest.mark.parametrize("adapters", [None, (3, 16, "both")])
def test_layer(T, fn, adapters):
    layer = Layer(T, 512, 256, 256, 16, 4, packed=True, adapters=adapters)
    beside(lambda s: layer.call(fn, stream=s), layer.call(fn))


def test_a_stream_of_another_kind():
    """Only the stream's pointer is asked for."""
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    layer = Layer(3, 512, 256, 256, 16, 4, packed=True)
    want = layer.call(moe.layer_forward)
    side.wait_stream(torch.cuda.current_stream())
    out = layer.call(moe.layer_forward, stream=Handle())
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
