"""Norms of rows whose squares, or their sum, do not fit fp32, against fp64: values up to the largest and down
to tiny ones, rows of both, one wave's columns far from the others'."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import plain_norms
from test_gpu_norms import check

pytestmark = pytest.mark.gpu

# widths of one wave a row, of four (some without columns in their last piece) and of eight
WIDTHS = [64, 520, 1032, 2048, 2056, 4096, 8192]


def rows(powers, d, seed):
    """One row for each power of two, of that standard deviation, no value past 3 of it."""
    v = plain.bf16((len(powers), d), 1.0, seed).clamp(-3, 3)
    return (v.double() * 2.0 ** torch.tensor(powers, dtype=torch.float64)[:, None]).bfloat16().cuda()


def ones(d, seed):
    return (1 + plain.bf16((d,), 0.2, seed)).cuda()


def with_ends(want, rows):
    """bf16 and fp32 hold fewer bits below 2^-126: half a step of bf16 there, and for a sum of fp32 one of each row."""
    return {n: (v, b + (rows * 2.0 ** -149 if n in ("dpre_weight", "dpost_weight") else 2.0 ** -134)) for n, (v, b) in want.items()}


def both(y, residual, s, eps, what):
    """Forward and backward against fp64.  scale is 1."""
    out, normed = moe.block_norms(y, residual, pre_weight=s["pre"], post_weight=s["post"], eps=eps)
    want = plain_norms.forward(y, residual, s["pre"], s["post"], None, 1.0, eps, out)
    check(dict(out=out, normed=normed), with_ends(want, len(y)), what)
    grads = moe.block_norms_backward(None, s["dnormed"], y, out, pre_weight=s["pre"], post_weight=s["post"], eps=eps)
    want = plain_norms.backward(None, s["dnormed"], y, out, s["pre"], s["post"], None, 1.0, eps)
    check(grads._asdict(), with_ends(want, len(y)), what)


def inputs(T, d):
    return dict(pre=ones(d, 2), post=ones(d, 3), dnormed=plain.bf16((T, d), 0.02, 6).cuda())


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("eps", [moe.NORM_EPS, 0.0])
def test_large_values(d, eps):
    powers = [0, 56, 57, 58, 59, 60, 62, 63, 64, 80, 110, 120, 125]
    y, residual = rows(powers, d, 11), rows(powers[::-1], d, 12)
    both(y, residual, inputs(len(powers), d), eps, (d, eps))


@pytest.mark.parametrize("d", WIDTHS)
def test_tiny_values_without_eps(d):
    powers = [0, -40, -48, -52, -56, -64, -75, -100]
    y, residual = rows(powers, d, 13), rows([p - 10 for p in powers], d, 14)
    s = inputs(len(powers), d)
    out, normed = moe.block_norms(y, residual, pre_weight=s["pre"], post_weight=s["post"], eps=0.0)
    check(dict(out=out, normed=normed), plain_norms.forward(y, residual, s["pre"], s["post"], None, 1.0, 0.0, out), d)
    same, normed = moe.block_norms(None, y, pre_weight=s["pre"], eps=0.0)
    check(dict(normed=normed), plain_norms.forward(None, y, s["pre"], None, None, 1.0, 0.0, y), d)
    grads = moe.block_norms_backward(None, s["dnormed"], None, y, pre_weight=s["pre"], eps=0.0)
    check(grads._asdict(), plain_norms.backward(None, s["dnormed"], None, y, s["pre"], None, None, 1.0, 0.0), d)


@pytest.mark.parametrize("d", [520, 2056, 4096, 8192])
@pytest.mark.parametrize("eps", [moe.NORM_EPS, 0.0])
def test_one_part_of_a_row_is_far_from_the_rest(d, eps):
    """A wave's columns (512 of 8 a lane) of another range than the others', zeros among them."""
    T, powers = 6, [(0, 70), (70, 0), (-60, 70), (-60, 0), (0, -60), (110, -110)]
    y = torch.cat([torch.cat([rows([a], 512, 20 + i), rows([b], d - 512, 30 + i)], 1) for i, (a, b) in enumerate(powers)])
    y[0, :512] = 0
    both(y, torch.zeros_like(y), inputs(T, d), eps, (d, eps))


def test_infinities_stay_in_their_row():
    """1 / rms is zero there: zeros, and NaN where the infinity was; a NaN takes its whole row."""
    for d in WIDTHS:
        x = rows([0, 3, 100, 2], d, 40)
        clean = moe.block_norms(None, x, pre_weight=ones(d, 2))[1]
        x[1, 5], x[3, d - 1] = float("inf"), float("nan")
        got = moe.block_norms(None, x, pre_weight=ones(d, 2))[1]
        assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
        assert got[1, 5].isnan() and not got[1, :5].any() and not got[1, 6:].any() and got[3].isnan().all()
