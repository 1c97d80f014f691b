"""Few tokens by outputs so wide that they take the large tiles: all but a few of a tile's rows do not exist."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import plain_ffn
from plain_int8 import product
from test_gpu_ffn import check, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,n_in,n_out", [(1, 256, 50001), (40, 128, 65536), (64, 1040, 49153), (3, 64, 163840), (70, 144, 57344)])
def test_linear_int8(T, n_in, n_out):
    W, ws = moe.quantize_int8(plain.bf16((n_out, n_in), 0.02, 2).cuda())
    q, xs = moe.quantize_int8(plain.bf16((T, n_in), 1.0, T).cuda())
    whole = torch.full((T * n_out + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = moe.linear_int8(q, W, ws, x_scale=xs, out=whole[:T * n_out].view(T, n_out))
    assert (whole[T * n_out:] == 7).all()  # rows that do not exist are not written
    v = product(q, xs, W, ws)
    off = (out.double() - v).abs() - v.abs() * (2.0 ** -8 + 4 * 2.0 ** -24)  # as in the test of the other sizes
    assert off.max() <= 0, off.max().item()


@pytest.mark.parametrize("T,d,F", [(20, 64, 32768), (64, 136, 24576), (9, 264, 28680)])
def test_gated_ffn(T, d, F):
    x, (wg, wu, wd) = plain.bf16((T, d), 1.0, T).cuda(), weights(d, F)
    gate, up = (torch.empty((T, F), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = moe.gated_ffn(x, wg, wu, wd, gate=gate, up=up)
    check(dict(out=out, gate=gate, up=up), plain_ffn.forward(x, wg, wu, wd), (T, d, F))
    dout = plain.bf16((T, d), 0.01, T + 1).cuda()
    got = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
    check(got._asdict(), plain_ffn.backward(dout, x, wg, wu, wd, gate, up), (T, d, F))


def test_widest_linear_int8():
    """The most columns that the call takes: 34 GB of codes."""
    n = 2 ** 31 - 256
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    W, ws = torch.zeros((n, 16), dtype=torch.int8, device="cuda"), torch.ones(n, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    q, xs = rand(2, 16), torch.tensor([0.5, 2.0], device="cuda")
    for part in (slice(0, 300), slice(2 ** 30 - 300, 2 ** 30 + 300), slice(n - 600, n)):
        W[part] = rand(part.stop - part.start, 16)
    out = moe.linear_int8(q, W, ws, x_scale=xs)
    for part in (slice(0, 600), slice(2 ** 30 - 600, 2 ** 30 + 600), slice(n - 1200, n)):
        v = product(q, xs, W[part], ws[part])
        assert ((out[:, part].double() - v).abs() <= v.abs() * 2.0 ** -8).all()
    del W, ws, out
    torch.cuda.empty_cache()
