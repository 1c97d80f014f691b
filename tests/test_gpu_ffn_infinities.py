"""An infinity or NaN among what gated_ffn_backward multiplies gives what the formula gives: that infinity with its
sign or NaN, in the results that it reaches, also where values are held in two halves of which one may be zero."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import plain_ffn
from test_gpu_ffn import weights

pytestmark = pytest.mark.gpu

# few tokens in halves, with K of dx split and whole, large and small tiles of the weights; one rounding
SIZES = [(1, 64, 72), (5, 256, 344), (33, 512, 136), (64, 264, 1000), (20, 1032, 4096), (40, 4096, 4104), (65, 128, 264), (200, 264, 512)]


def same_class(got, want, what):
    """Finite where the formula is; the same infinity where it is infinite; NaN where it is NaN."""
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    assert torch.equal(got.isnan(), want.isnan()), what
    at = torch.isinf(want)
    assert torch.equal(got[at], want[at]), what


def setup(T, d, F):
    x, dout = plain.bf16((T, d), 1.0, T).cuda(), plain.bf16((T, d), 0.5, T + 1).cuda()
    gate, up = plain.bf16((T, F), 1.5, 7).cuda(), plain.bf16((T, F), 1.0, 8).cuda()
    # halves that are zero: a = 0.5 g s u of s = 1/2 and u a power of two has none left over
    gate[:, ::5], up[:, ::3] = 0.0, 2.0
    up[up == 0] = 1.0  # 0 times an infinity is NaN in the formula and not the subject
    return [dout, x, *weights(d, F), gate, up]


@pytest.mark.parametrize("T,d,F", SIZES)
def test_infinity_in_dout(T, d, F):
    """dw_down = dout^T a, and every other channel of it."""
    args = setup(T, d, F)
    clean = moe.gated_ffn_backward(*args)
    args[0][T // 2, 3], args[0][0, d - 1] = float("inf"), float("-inf")
    got = moe.gated_ffn_backward(*args)
    g, u = args[5].double(), args[6].double()
    a = (g * plain_ffn.sigmoid(g) * u).bfloat16().double()  # zeros of a gate of 0 stay zeros
    want = sum(args[0][t].double()[:, None] * a[t] for t in range(T))  # a product's own way with 0 times an infinity
    same_class(got.dw_down, want, "dw_down")
    rest = [c for c in range(d) if c not in (3, d - 1)]
    assert torch.equal(got.dw_down[rest], clean.dw_down[rest])


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,d,F", SIZES)
def test_infinity_in_x(T, d, F, value):
    """dw_gate = dG^T x and dw_up = dU^T x: one column of each."""
    args = setup(T, d, F)
    clean = moe.gated_ffn_backward(*args)
    args[1][T // 2, 5] = value
    got = moe.gated_ffn_backward(*args)
    assert torch.equal(got.dx, clean.dx) and torch.equal(got.dw_down, clean.dw_down)
    dout, g, u, wd = args[0].double(), args[5].double(), args[6].double(), args[4].double()
    s, dA = plain_ffn.sigmoid(g), dout @ wd
    dU, dG = dA * g * s, dA * u * s * (1 + g * (1 - s))
    for name, v in (("dw_up", dU), ("dw_gate", dG)):
        same_class(getattr(got, name)[:, 5], v[T // 2] * value, name)
        rest = [c for c in range(d) if c != 5]
        assert torch.equal(getattr(got, name)[:, rest], getattr(clean, name)[:, rest]), name


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,d,F", SIZES)
def test_infinity_in_weights(T, d, F, value):
    """dx = dG w_gate + dU w_up: one column of it for each matrix."""
    args = setup(T, d, F)
    clean = moe.gated_ffn_backward(*args)
    f = F - 1 if (F - 1) % 5 else F - 2  # where the gate is not 0
    args[2][f, 1], args[3][f, d - 2] = value, value
    got = moe.gated_ffn_backward(*args)
    for a, b in zip(got[1:], clean[1:]):
        assert torch.equal(a, b)
    dout, g, u, wd = args[0].double(), args[5].double(), args[6].double(), args[4].double()
    s, dA = plain_ffn.sigmoid(g), dout @ wd
    dU, dG = dA * g * s, dA * u * s * (1 + g * (1 - s))
    same_class(got.dx[:, 1], dG[:, f] * value, "w_gate")
    same_class(got.dx[:, d - 2], dU[:, f] * value, "w_up")
    rest = [c for c in range(d) if c not in (1, d - 2)]
    assert torch.equal(got.dx[:, rest], clean.dx[:, rest])
