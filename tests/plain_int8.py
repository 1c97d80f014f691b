"""The quantiser and the 8-bit projection by whole numbers, for their tests."""
import numpy as np
import torch


def codes(x):
    """(q, scale) of finite bf16 rows on the CPU.  127 |x| = q top + rest with whole q, all exact in
    fp64 (8, 8 and 7 bits); rounded up past half of top, and on it to the even q."""
    v = x.double()
    top = v.abs().amax(1, keepdim=True)
    t, d = 127.0 * v.abs(), torch.where(top > 0, top, torch.ones_like(top))
    q = torch.floor(t / d)
    rest = t - q * d
    low = rest < 0  # the quotient was rounded up to a whole number
    q, rest = torch.where(low, q - 1, q), torch.where(low, rest + d, rest)
    q = q + ((2 * rest > d) | ((2 * rest == d) & (q % 2 != 0)))
    scale = top[:, 0].float().numpy() / np.float32(127)
    return torch.where(v < 0, -q, q).to(torch.int8), scale


def product(q, xs, W, ws):
    """The projection's value in fp64 (whole sums below 2^53)."""
    return (q.double() @ W.double().T) * xs.double()[:, None] * ws.double()
