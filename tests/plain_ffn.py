"""The dense gated block and its gradients in fp64, with bounds on what a bf16 call may be off.

Bounds count roundings: one to bf16 is off by at most 2^-8 of the value, and a sum of K products
on the matrix cores by at most (K / 32 + 10) 2^-23 of the sum of the products' absolute values (a
step of 32 rounds once, within 2^-23 of the running sum; joins of split sums are among the 10).
An error on the way passes through the next product with that product's absolute values, times
two: a bound's own second-order terms, of 2^-8 of it, stay far below that.  What lies below 2^-126,
the least normal fp32 and bf16 value, may be flushed to zero by the matrix cores or the hardware's
2^x: each factor may lose that much, and so may the result."""
import torch

H = 2.0 ** -8  # half a step of bf16, relative
LEAST = 2.0 ** -126


def mat(a, b):
    return a.double() @ b.double()


def sum_bound(K):
    return (K / 32 + 10) * 2.0 ** -23



def sigmoid(g):
    return 1.0 / (1.0 + torch.exp(-g))


def forward(x, wg, wu, wd, inner=H):
    """{name: (value, bound)} of out, gate, up; inner: what a's rounding may leave, relative."""
    d, F = wg.shape[1], wg.shape[0]
    g, u = mat(x, wg.T), mat(x, wu.T)
    dg = mat(x.abs(), wg.abs().T) * sum_bound(d)
    du = mat(x.abs(), wu.abs().T) * sum_bound(d)
    s = g * sigmoid(g)
    a = s * u
    # |silu'| <= 1.1; silu and the product in fp32: 16 ulps
    da = 2 * (1.1 * dg * u.abs() + s.abs() * du) + a.abs() * (inner + 2.0 ** -20)
    out = mat(a, wd.T)
    dout = 2 * mat(da + LEAST, wd.abs().T) + LEAST + mat(a.abs(), wd.abs().T) * 2 * sum_bound(F) + out.abs() * H
    return dict(out=(out, dout), gate=(g, dg + g.abs() * H), up=(u, du + u.abs() * H))


def backward(dout, x, wg, wu, wd, g, u, inner=H):
    """{name: (value, bound)} of the gradients, g and u the kept bf16 projections; inner: what the roundings
    of a, dG and dU may leave, relative."""
    T, d = x.shape
    F = wg.shape[0]
    g, u, x, dout = g.double(), u.double(), x.double(), dout.double()
    dA = mat(dout, wd)
    eA = mat(dout.abs(), wd.abs()) * sum_bound(d)
    s = sigmoid(g)
    fg, fu = u * s * (1 + g * (1 - s)), g * s
    a = g * s * u
    # the factors in fp32: s within 8 ulps (1 - s absolutely, times g up to 88), then the rounding;
    # 1 + g (1 - s) may cancel, so its error counts against 1 + |g|
    dG, dU = dA * fg, dA * fu
    eG = 2 * eA * fg.abs() + dG.abs() * inner + 2 * dA.abs() * u.abs() * s * (1 + g.abs()) * 2.0 ** -19
    eU = 2 * eA * fu.abs() + dU.abs() * inner + 2 * dU.abs() * 2.0 ** -19
    ea = a.abs() * (inner + 2.0 ** -19)

    def product(terms, K):
        v = sum(mat(p, q) for p, _, q in terms)
        e = sum(2 * mat(ep + LEAST, q.abs()) + mat(p.abs(), q.abs()) * 2 * sum_bound(K) for p, ep, q in terms)
        return v, e + v.abs() * H + LEAST

    return dict(dx=product([(dG, eG, wg.double()), (dU, eU, wu.double())], 2 * F),
                dw_gate=product([(dG.T, eG.T, x)], T), dw_up=product([(dU.T, eU.T, x)], T),
                dw_down=tuple(t.T for t in product([(a.T, ea.T, dout)], T)))
