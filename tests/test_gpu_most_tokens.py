"""2^24 tokens, the most that the calls take: rows around each launch's first and last ones have what a call
of those rows alone gives."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain

pytestmark = pytest.mark.gpu

T = 1 << 24
PARTS = [slice(0, 70), slice((1 << 23) - 70, (1 << 23) + 70), slice(T - 70, T)]


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def values(d, std=1.0, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)


def test_quantize_and_linear_int8():
    x = values(16)
    q, scale = moe.quantize_int8(x)
    W, w_scale = moe.quantize_int8(plain.bf16((24, 16), 1.0, 3).cuda())
    whole, coded = moe.linear_int8(x, W, w_scale), moe.linear_int8(q, W, w_scale, x_scale=scale)
    assert torch.equal(whole, coded)
    for part in PARTS:
        a, b = moe.quantize_int8(x[part])
        assert torch.equal(q[part], a) and torch.equal(scale[part], b)
        assert torch.equal(whole[part], moe.linear_int8(x[part], W, w_scale))


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_norms_of_narrow_rows(gate):
    y, residual, pre, post = values(8), values(8, seed=2), plain.bf16((8,), 1.0, 3).cuda(), plain.bf16((8,), 1.0, 4).cuda()
    g = values(8, seed=5) if gate == "token" else plain.bf16((8,), 1.0, 5).cuda()
    kw = dict(pre_weight=pre, post_weight=post)
    out, normed = moe.block_norms(y, residual, gate=g, **kw)
    grads = moe.block_norms_backward(residual, y, y, out, gate=g, **kw)
    for part in PARTS:
        gp = g[part] if gate == "token" else g
        a, b = moe.block_norms(y[part], residual[part], gate=gp, **kw)
        assert torch.equal(out[part], a) and torch.equal(normed[part], b)
        c = moe.block_norms_backward(residual[part], y[part], y[part], a, gate=gp, **kw)
        assert torch.equal(grads.dresidual[part], c.dresidual) and torch.equal(grads.dy[part], c.dy)


def test_norms_of_rows_of_a_block():
    """The narrowest rows that take a block each: 69 GB of them."""
    d = 2056
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of device memory")
    x, pre = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda"), plain.bf16((d,), 1.0, 3).cuda()
    for i, part in enumerate(PARTS):
        x[part] = plain.bf16((part.stop - part.start, d), 1.0, 4 + i).cuda()
    normed = moe.block_norms(None, x, pre_weight=pre)[1]
    for part in PARTS:
        assert torch.equal(normed[part], moe.block_norms(None, x[part], pre_weight=pre)[1])
    del x
    # y and the stream in place, a gate of each token
    for part in PARTS:
        rows = plain.bf16((part.stop - part.start, d), 1.0, 9).cuda()
        normed[part] = rows
    y = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    y[PARTS[1]] = 2
    out = moe.block_norms(y, normed, post_weight=pre, gate=y, out=normed)[0]
    for part in PARTS:
        rows = plain.bf16((part.stop - part.start, d), 1.0, 9).cuda()
        assert torch.equal(out[part], moe.block_norms(y[part], rows, post_weight=pre, gate=y[part])[0])
