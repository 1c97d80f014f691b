"""The 8-bit projection and its quantiser against whole-number forms: every tile that the sizes
choose, ties, rows of every magnitude and kind, streams and captured graphs."""
import numpy as np
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
from plain_int8 import codes, product

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def rows(T, n, seed):
    """Rows of magnitudes from 2^-130 to 2^126, some with many ties (halves of the largest), one of zeros."""
    x = plain.bf16((T, n), 1.0, seed).float()
    x = x * torch.exp2(torch.linspace(-130, 124, T).round())[:, None]
    x[T // 2] = 0
    x = x.bfloat16()
    x[0, : n // 2] = x[0, -1] / 2
    return x


# a row's pieces within one round of its block, just past a round, longer than the registers hold
@pytest.mark.parametrize("T,n", [(1, 16), (5, 48), (64, 2048), (33, 2064), (9, 7168), (4, 8192), (5, 8208), (3, 65536), (1000, 112)])
def test_quantize(T, n):
    x = rows(T, n, T + n)
    q, scale = moe.quantize_int8(x.cuda())
    want_q, want_s = codes(x)
    assert torch.equal(q.cpu(), want_q)
    assert np.array_equal(scale.cpu().numpy(), want_s)


def test_every_code_and_tie():
    """Each bf16 value against each largest value of one binade: every quotient that a row can hold."""
    for top in range(0x4300, 0x4380):  # 128 to 255
        x = torch.arange(0x3E00, top + 1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
        x = torch.cat([x, -x, torch.zeros(-2 * len(x) % 16, dtype=torch.bfloat16)])[None]
        q, _ = moe.quantize_int8(x.cuda())
        assert torch.equal(q.cpu(), codes(x)[0]), hex(top)


def test_rows_that_are_not_finite():
    x = plain.bf16((6, 160), 1.0, 1)
    x[1, 3], x[2, 159], x[4, 0] = float("inf"), float("nan"), float("-inf")
    q, scale = moe.quantize_int8(x.cuda())
    want, s = codes(x[[0, 3, 5]])
    assert torch.equal(q.cpu()[[0, 3, 5]], want) and np.array_equal(scale.cpu().numpy()[[0, 3, 5]], s)
    assert not q[[1, 2, 4]].any() and torch.isnan(scale[[1, 2, 4]]).all()
    W = torch.randint(-127, 128, (40, 160), dtype=torch.int8, device="cuda")
    out = moe.linear_int8(x.cuda(), W, torch.ones(40, device="cuda"))
    assert torch.isnan(out[[1, 2, 4]]).all() and torch.isfinite(out[[0, 3, 5]]).all()


# tokens, inner and outer widths: the few-token tiles, widths that end inside a tile, outer widths
# that are no multiple of anything, splits of the inner width, the large tiles
CASES = [(1, 16, 1), (1, 7168, 3584), (5, 64, 33), (16, 3584, 7168), (32, 208, 130), (33, 4096, 1000), (48, 7168, 3584),
         (64, 1040, 65), (65, 128, 127), (100, 8192, 96), (257, 3584, 515), (1000, 2048, 2049), (1021, 7168, 320),
         (300, 4096, 264), (4096, 272, 4100), (3001, 3584, 7168)]


@pytest.mark.parametrize("T,n_in,n_out", CASES)
def test_linear(T, n_in, n_out):
    x, w = plain.bf16((T, n_in), 1.0, T).cuda(), plain.bf16((n_out, n_in), 0.02, 2).cuda()
    W, ws = moe.quantize_int8(w)
    q, xs = moe.quantize_int8(x)
    out = moe.linear_int8(x, W, ws)
    v = product(q, xs, W, ws)
    # two fp32 products and the sum's way to fp32, then the rounding
    off = (out.double() - v).abs() - v.abs() * (H + 4 * 2.0 ** -24)
    assert off.max() <= 0, off.max().item()
    assert torch.equal(out, moe.linear_int8(q, W, ws, x_scale=xs))


@pytest.mark.parametrize("T,n_in,n_out", [(3, 65536, 24), (40, 65536, 40), (300, 65536, 136)])
def test_longest_sums(T, n_in, n_out):
    """All codes at their ends: sums next to 2^30, exact."""
    q = torch.full((T, n_in), -128, dtype=torch.int8, device="cuda")
    W = torch.full((n_out, n_in), -128, dtype=torch.int8, device="cuda")
    W[1::2] = 127
    one = lambda n: torch.ones(n, device="cuda")
    out = moe.linear_int8(q, W, one(n_out), x_scale=one(T))
    want = torch.where(torch.arange(n_out) % 2 == 0, 128.0 * 128 * 65536, -128.0 * 127 * 65536).bfloat16().cuda()
    assert torch.equal(out, want.expand(T, -1))


def test_no_tokens():
    W, ws = torch.zeros((8, 16), dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    assert moe.linear_int8(x, W, ws).shape == (0, 8)
    q, s = moe.quantize_int8(x)
    assert q.shape == (0, 16) and s.shape == (0,) and moe.linear_int8(q, W, ws, x_scale=s).shape == (0, 8)


@pytest.mark.parametrize("T,n_in,n_out", [(5, 160, 33), (48, 4096, 90), (300, 1040, 1023)])
def test_graph_streams_and_bounds(T, n_in, n_out):
    """Replays and a side stream give the eager bits, and nothing is written past the outputs."""
    x = plain.bf16((T, n_in), 1.0, 1).cuda()
    W, ws = moe.quantize_int8(plain.bf16((n_out, n_in), 0.02, 2).cuda())
    work = torch.full((moe.linear_int8_workspace_size(T, n_in, n_out),), 255, dtype=torch.uint8, device="cuda")
    whole = torch.full((T * n_out + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = whole[2048: 2048 + T * n_out].view(T, n_out)
    call = lambda: moe.linear_int8(x, W, ws, out=out, workspace=work)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (5, 6, 7):
        x.copy_(plain.bf16((T, n_in), 1.0, seed))
        want = moe.linear_int8(x, W, ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = moe.linear_int8(x, W, ws, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        out.zero_()
        work.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert (whole[:2048] == 7).all() and (whole[2048 + T * n_out:] == 7).all()


def test_offsets_past_31_bits():
    """Results that begin past 2^31 values, and codes of a token past them."""
    T, n_in, n_out, n = 40000, 16, 65536, 100
    q = torch.randint(-127, 128, (T, n_in), dtype=torch.int8, device="cuda")
    W = torch.randint(-127, 128, (n_out, n_in), dtype=torch.int8, device="cuda")
    one = lambda k: torch.ones(k, device="cuda")
    out = moe.linear_int8(q, W, one(n_out), x_scale=one(T))
    for rows in (slice(0, n), slice(T - n, T)):
        assert torch.equal(out[rows], (q[rows].double() @ W.double().T).bfloat16())
    T, n_in = 40000, 65536
    x = torch.zeros((T, n_in), dtype=torch.bfloat16, device="cuda")
    x[-n:] = plain.bf16((n, n_in), 1.0, 3).cuda()
    q, s = moe.quantize_int8(x)
    want_q, want_s = moe.quantize_int8(x[-n:].contiguous())
    assert torch.equal(q[-n:], want_q) and torch.equal(s[-n:], want_s) and not q[:-n].any()
