"""Gradients of the dense block where silu and its slope are tiny and what they meet is large: single products
with ones, so each result is one value of a formula."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain_ffn

pytestmark = pytest.mark.gpu


def bound(v, size, factor, inner):
    """In fp32, e^-|g| is taken of an argument of up to 145 that is rounded (2^-17 of the result), by the
    hardware's 2^x, and meets its reciprocal and some products: 2^-16 of the terms' sizes.  A factor below
    2^-126 is off by four roundings of 2^-150 at most, 4 2^-149 says more, and meets what `factor` says.
    Then come the rounding to bf16 (inner), the result's own, and what a value below 2^-126 may lose."""
    e = size * 2.0 ** -16 + factor * 4 * 2.0 ** -149
    return (e + (v.abs() + e) * (inner + plain_ffn.H)) * 1.01 + 4 * plain_ffn.LEAST


@pytest.mark.parametrize("T", [1, 64, 65, 200])
@pytest.mark.parametrize("least,most,u_power,d_power", [(-100, -80, 100, 60), (-100, -80, 60, 100), (-100, 100, 0, 100)])
def test_far_gates(T, least, most, u_power, d_power):
    """One row of w_down is ones and dout has one column, so dA is a power of two; the other weights are unit
    vectors or zeros, so dx is dU or dG; x is a unit vector of the first token, so the weights' gradients
    are that token's."""
    d = F = 256
    g = torch.linspace(least, most, F * T, dtype=torch.float64)[torch.randperm(F * T, generator=torch.Generator().manual_seed(1))]
    gate = g.view(T, F).to(torch.bfloat16).cuda()
    up = torch.full((T, F), 2.0 ** u_power).to(torch.bfloat16).cuda()
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    dout, w_down, x = zeros(T, d), zeros(d, F), zeros(T, d)
    dout[:, 0], w_down[0], x[0, 0] = 2.0 ** d_power, 1.0, 1.0
    eye, zero = torch.eye(F, d).to(torch.bfloat16).cuda(), zeros(F, d)

    gd, u, dA = gate.double(), 2.0 ** u_power, 2.0 ** d_power
    s, one = plain_ffn.sigmoid(gd), plain_ffn.sigmoid(-gd)  # and 1 - s, without its cancellation
    a, dU, dG = gd * s * u, dA * gd * s, dA * u * s * (1 + gd * one)
    # up to 64 tokens in two halves of bf16
    inner = 2.0 ** -16 if T <= 64 else plain_ffn.H
    eU, eG = bound(dU, dU.abs(), dA, inner), bound(dG, dA * u * s * (1 + gd.abs() * one), dA * u, inner)

    def check(got, want, e, what):
        off = (got.double() - want).abs() - e
        assert off.max() <= 0, (what, off.max().item(), want.flatten()[off.argmax()].item(), got.flatten()[off.argmax()].item())

    for w_gate, w_up, v, e in ((zero, eye, dU, eU), (eye, zero, dG, eG)):
        got = moe.gated_ffn_backward(dout, x, w_gate, w_up, w_down, gate, up)
        check(got.dx, v, e, "dx")
        check(got.dw_up[:, 0], dU[0], eU[0], "dw_up")
        check(got.dw_gate[:, 0], dG[0], eG[0], "dw_gate")
        if T == 1:
            # here a is a factor of the product with dout: each of its two halves, where it lies below 2^-126, may
            # be flushed by the matrix cores, which is up to 2^-126 dA in the result
            e = bound(dA * a, (dA * a).abs(), dA * u, inner) + 2 * plain_ffn.LEAST * dA
            check(got.dw_down[0], dA * a[0], e[0], "dw_down")
