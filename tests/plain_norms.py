"""The step between two blocks and its gradients in fp64, with bounds on what a call may be off.

Bounds count roundings: one to bf16 is off by at most H = 2^-8 of the value.  In fp32, a row's sum
of up to 8192 terms (32 of a lane one after another, then a tree and at most eight waves) is off by
at most 48 2^-24 of the sum of the absolute values, a statistic from it by half of that and a few
roundings more, and each product adds one: E = 2^-18 covers each such chain.  A sum over tokens
adds one rounding for each row of a thread and each join."""
import torch

H, E = 2.0 ** -8, 2.0 ** -18


def norm(v, eps):
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    return v * r, r


def forward(y, residual, pre, post, gate, scale, eps, got_out):
    """{name: (value, bound)} of out, and of normed of the out that the call gave."""
    found = {}
    if y is not None:
        v = y.double()
        if post is not None:
            v = norm(v, eps)[0] * post.double()
        v = scale * v * (1.0 if gate is None else gate.double())
        out = residual.double() + v
        found["out"] = (out, out.abs() * H + (v.abs() + residual.double().abs()) * E)
    if pre is not None:
        n = norm(got_out.double(), eps)[0] * pre.double()
        found["normed"] = (n, n.abs() * (H + E))
    return found


def backward(dout, dnormed, y, out, pre, post, gate, scale, eps):
    """{name: (value, bound)} of the gradients."""
    zero = torch.zeros_like(dout if dout is not None else dnormed, dtype=torch.float64)
    T = zero.shape[0]
    S = (T / 256 + 48) * 2.0 ** -24  # a sum over the tokens
    found = {}
    G = zero + (0 if dout is None else dout.double())
    eG = G.abs() * E
    if pre is not None:
        rh, ir = norm(out.double(), eps)
        dn = zero + (0 if dnormed is None else dnormed.double())
        e = dn * pre.double()
        mean, size = (e * rh).mean(1, keepdim=True), (e * rh).abs().mean(1, keepdim=True)
        G = G + ir * (e - rh * mean)
        eG = eG + ir * (e.abs() + rh.abs() * size) * E
        found["dpre_weight"] = ((dn * rh).sum(0), (dn * rh).abs().sum(0) * (E + S))
    found["dresidual"] = (G, eG + G.abs() * H)
    if y is None:
        return found
    yh, iy = norm(y.double(), eps) if post is not None else (y.double(), 1.0)
    w = post.double() if post is not None else 1.0
    g = gate.double() if gate is not None else 1.0
    if gate is not None:
        dg, eg = scale * G * yh * w, abs(scale) * (eG + G.abs() * E) * (yh * w).abs()
        found["dgate"] = (dg.sum(0), eg.sum(0) + dg.abs().sum(0) * S) if gate.dim() == 1 else (dg, eg + dg.abs() * H)
    b, eb = scale * G * g, abs(scale) * (eG + G.abs() * E) * (g.abs() if gate is not None else 1.0)
    if post is None:
        found["dy"] = (b, eb + b.abs() * H)
        return found
    found["dpost_weight"] = ((b * yh).sum(0), ((eb + b.abs() * E) * yh.abs()).sum(0) + (b * yh).abs().sum(0) * S)
    f, ef = b * w, (eb + b.abs() * E) * w.abs()
    mean, size = (f * yh).mean(1, keepdim=True), (f * yh).abs().mean(1, keepdim=True)
    em = (ef * yh.abs()).mean(1, keepdim=True) + size * E
    dy = iy * (f - yh * mean)
    found["dy"] = (dy, iy * (ef + yh.abs() * em + (f.abs() + yh.abs() * size) * E) + dy.abs() * H)
    return found
