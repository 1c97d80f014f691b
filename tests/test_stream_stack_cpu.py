"""What LayerStack refuses before anything runs, for stacks with dense layers."""
import pytest
import torch

from mxfp4_expert_gemm_amd.stream import LayerStack


def dense(d=64, F=72):
    b = lambda *shape: torch.empty(shape, dtype=torch.bfloat16)
    return dict(w_gate=b(F, d), w_up=b(F, d), w_down=b(d, F))


def test_dense_stack_refusals():
    stack = LayerStack([dense(), dense(F=128)], 0, 0, 1, 4, device="cpu")
    assert stack.widths == [64, 64] and stack.resident == [None, None]
    assert stack.workspace is None and stack.slots is None
    x = torch.empty(4, 64, dtype=torch.bfloat16)
    norm = torch.empty(64, dtype=torch.bfloat16)
    head = (torch.empty(32, 64, dtype=torch.int8), torch.empty(32))
    for bad in (dict(x=x[:3]), dict(x=x[:, :56]), dict(x=x.float()), dict(x=x, head=head),
                dict(x=x, final_norm=norm, head=torch.empty(32, 72, dtype=torch.bfloat16)),
                dict(x=x, final_norm=norm, head=torch.empty(32, 64))):
        with pytest.raises(ValueError):
            stack.forward(**bad)
    with pytest.raises(ValueError):
        stack.forward_layer(0, x, routing={})
    with pytest.raises(ValueError):
        stack.step([x])
    with pytest.raises(ValueError):
        LayerStack([dense()], 0, 0, 2, 4, device="cpu")
    for bad in (norm[:32], norm.float()):
        first = LayerStack([dict(dense(), pre_norm=bad)], 0, 0, 0, 4, device="cpu")
        with pytest.raises(ValueError):
            first.forward(x)
    two = LayerStack([dense(), dense(d=72)], 0, 0, 0, 4, device="cpu")
    with pytest.raises(ValueError):
        two.forward(x)
    with pytest.raises(ValueError):  # a routed layer's experts are pinned host memory
        LayerStack([dense(), dict(router_w=torch.empty(4, 64), expert_blob_host=torch.empty(8, dtype=torch.uint8))],
                   1, 64, 1, 4, device="cpu")
