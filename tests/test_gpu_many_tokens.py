"""Token counts past the second dimension of one grid, on widths that the matrix cores do not take (n_in
no multiple of 64): every row as in a small call on the same rows."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
from test_gpu_lora import dev_lora

pytestmark = pytest.mark.gpu
BASE = 4096


@pytest.mark.parametrize("T", [262140, 262141, 524301, 1 << 24])
def test_projection(T):
    n_in, n_out, N, R = 32, 7, 3, 8
    x, W = plain.bf16((BASE, n_in), 1.0, 1).cuda(), plain.bf16((n_out, n_in), 0.2, 2).cuda()
    lo = plain.adapters(N, R, n_in, n_out, 3)
    ids = torch.arange(BASE, dtype=torch.int32) % (N + 1) - 1
    few = moe.linear_lora(x, W, dev_lora(lo, ids))
    few0 = moe.linear_bf16(x, W)
    over = (T + BASE - 1) // BASE
    big = x.repeat(over, 1)[:T]
    got = moe.linear_lora(big, W, dev_lora(lo, ids.repeat(over)[:T]))
    assert torch.equal(got, few.repeat(over, 1)[:T])
    assert torch.equal(moe.linear_bf16(big, W), few0.repeat(over, 1)[:T])
