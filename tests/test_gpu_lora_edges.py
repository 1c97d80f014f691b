"""linear_lora where the adapter's term cancels, overflows bf16 or holds infinities: every kernel the
sizes choose gives what the formula gives."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe

pytestmark = pytest.mark.gpu

# T, n_in, n_out: the GEMV, the small tiles, the grouped first product, and the matrix cores below
# 32 tokens, which large matrices take
SHAPES = [(3, 64, 40), (40, 64, 40), (600, 64, 40), (7, 7168, 3584), (700, 64, 8200)]


def small_lora(T, n_in, n_out, N=2, R=8):
    """Zero adapters, every other token naming adapter 1."""
    return (torch.zeros((N, R, n_in)), torch.zeros((N, n_out, R)), torch.arange(T, dtype=torch.int32) % N)


def run(x, W, a, b, ids):
    lo = moe.Lora(a.bfloat16().cuda(), b.bfloat16().cuda(), torch.ones(a.shape[0]).cuda(), ids.cuda())
    return moe.linear_lora(x.bfloat16().cuda(), W.bfloat16().cuda(), lo).float().cpu()


@pytest.mark.parametrize("T,n_in,n_out", SHAPES)
def test_a_term_that_cancels(T, n_in, n_out):
    """u = (2^20 + 2^10 + 1, 2^20 + 2^10), exact in fp32, against b = (1, -1): the output is 1."""
    x, W = torch.zeros((T, n_in)), torch.zeros((n_out, n_in))
    a, b, ids = small_lora(T, n_in, n_out)
    x[:, :3] = torch.tensor([2.0 ** 10, 2.0 ** 5, 1.0])
    a[1, 0, :3] = x[0, :3]
    a[1, 5, :3] = torch.tensor([2.0 ** 10, 2.0 ** 5, 0.0])
    b[1, :, 0], b[1, :, 5] = 1.0, -1.0
    out = run(x, W, a, b, ids)
    assert (out[ids == 1] == 1.0).all() and (out[ids == 0] == 0.0).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T,n_in,n_out", SHAPES)
def test_u_between_the_largest_bf16_and_fp32(T, n_in, n_out, sign):
    """u = 2^127 (2 - 2^-10), which no bf16 value but infinity is near, times b = 2^-120."""
    x, W = torch.zeros((T, n_in)), torch.zeros((n_out, n_in))
    a, b, ids = small_lora(T, n_in, n_out)
    x[:, :2] = torch.tensor([2.0 ** 64, 2.0 ** 56])
    a[1, 2, :2] = sign * torch.tensor([2.0 ** 63 * (2 - 2.0 ** -7), 2.0 ** 71 * (2.0 ** -7 - 2.0 ** -10)])
    b[1, :, 2] = 2.0 ** -120
    u = float(x[0].double() @ a[1, 2].double())
    assert abs(u) == 2.0 ** 127 * (2 - 2.0 ** -10)
    want = torch.tensor(u * 2.0 ** -120).bfloat16().float()  # 2^8 (1 - 2^-11), rounded to 2^8
    out = run(x, W, a, b, ids)
    assert (out[ids == 1] == want).all() and (out[ids == 0] == 0.0).all()


@pytest.mark.parametrize("T,n_in,n_out", SHAPES)
def test_infinities_in_the_second_matrix(T, n_in, n_out):
    """Infinite entries of b times a u that bf16 holds exactly, that needs more bits of either sign,
    and that is zero; both infinities in one sum; a NaN.  Value, sign and class as the formula's."""
    inf, nan = float("inf"), float("nan")
    x, W = torch.zeros((T, n_in)), torch.zeros((n_out, n_in))
    x[:, :2] = torch.tensor([2.0 ** 10, 1.0])
    W[:, 1] = 0.5
    a, b, ids = small_lora(T, n_in, n_out)
    a[1, :5, :2] = torch.tensor([[0.0, 4.0], [1.0, 3.0], [-1.0, 3.0], [1.0, -3.0], [0.0, 0.0]])  # 4, 1027, -1021, 1021, 0
    rows = [[inf, 1, 0, 0, 0], [0, inf, 1, 0, 0], [0, 1, inf, 0, 0], [0, 0, 0, inf, 0], [1, 0, 0, 0, inf],
            [0, -inf, 0, 0, 0], [0, inf, -inf, 0, 0], [0, inf, inf, 0, 0], [nan, 1, 0, 0, 0], [1, 1, 1, 1, 0]]
    b[1, :, :5] = torch.tensor(rows, dtype=torch.float32)[torch.arange(n_out) % len(rows)]
    # 4 inf; 1027 inf; -1021 inf; 1021 inf; 0 inf; -1027 inf; 1027 inf + -1021 -inf; 1027 inf - 1021 inf; NaN; the sum
    want = torch.tensor([inf, inf, -inf, inf, nan, -inf, inf, nan, nan, 0.5 + 4 + 1027 - 1021 + 1021]).bfloat16().float()
    want = want[torch.arange(n_out) % len(rows)]
    out = run(x, W, a, b, ids)
    for t in range(T):
        if ids[t] == 1:
            assert torch.equal(out[t].isnan(), want.isnan()), t
            assert torch.equal(torch.nan_to_num(out[t], 7.0), torch.nan_to_num(want, 7.0)), t
        else:
            assert (out[t] == 0.5).all()
