"""Plain fp64 forms of the adapter projection and of the whole layer, for the tests of both.

They share no code with the library: a projection is a matrix product, an adapter is added to
the rows that name it, an expert's weights are decoded one formula at a time.
"""
import numpy as np
import torch


def bf16(shape, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float32) * std).bfloat16()


def adapters(N, R, n_in, n_out, seed, std=1.0):
    """A stack of adapters whose term is about as large as the projection's."""
    g = torch.Generator().manual_seed(seed + 7)
    return dict(a=bf16((N, R, n_in), std * n_in ** -0.5, seed), b=bf16((N, n_out, R), 0.2, seed + 1),
                scale=0.5 + torch.rand(N, generator=g))


def linear(x, W, lo=None, ids=None, rank=None):
    """(value, S): the projection with adapters in fp64, and the same sum over the products'
    absolute values, which the bounds on fp32 sums are relative to."""
    x, W = x.double(), W.double()
    v, s = x @ W.T, x.abs() @ W.abs().T
    if lo is not None:
        N, R = lo["a"].shape[:2]
        for i in range(N):
            r = R if rank is None else max(0, min(int(rank[i]), R))
            rows = (ids == i).nonzero()[:, 0]
            A, B = lo["a"][i, :r].double(), lo["b"][i, :, :r].double()
            sc = float(lo["scale"][i])
            if r and len(rows):
                v[rows] += sc * ((x[rows] @ A.T) @ B.T)
                s[rows] += sc * ((x[rows].abs() @ A.abs().T) @ B.abs().T)
    return v, s


def linear_bound(v, S, n_in):
    """How far a bf16 result may be from v: one rounding (2^-8 relative), fp32 sums of K
    products in matrix-core steps of 32 (a step adds at most its own rounding of 2^-23 of S,
    n_in / 32 steps for the projection, as many for u, and at most 8 + 34 more for the second
    product and the joins), and u's 16 bits in the second product (2^-16)."""
    return 2.0 ** -8 * v.abs() + S * ((2 * n_in / 32 + 42) * 2.0 ** -23 + 2.0 ** -16)


def round_bf16(v):
    return v.float().bfloat16().double()


def mxfp8(v):
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 8, torch.full_like(top, -127.0))
    e = e.clamp(-127, 127)
    q = (b / torch.exp2(e)).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step * torch.exp2(e)).reshape(v.shape)


def expert(blob, e, L, F):
    """fp64 gate, up and down of record e of a blob of checkpoint records (numpy uint8)."""
    n = F * L // 2 + F * L // 32
    rec = blob[3 * n * e: 3 * n * (e + 1)]
    out = []
    for m, (R, K) in enumerate(((F, L), (F, L), (L, F))):
        part = rec[m * n: (m + 1) * n]
        codes = part[: R * K // 2].reshape(R, K // 2)
        code = np.stack((codes & 15, codes >> 4), -1).reshape(R, K).astype(np.int64)
        ex, man = (code >> 1) & 3, code & 1
        mag = np.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (ex - 1.0))
        scale = 2.0 ** (part[R * K // 2:].reshape(R, K // 32).astype(np.float64) - 127)
        out.append(torch.from_numpy(np.where(code >= 8, -mag, mag) * np.repeat(scale, 32, 1)))
    return out


def layer(x, router_w, latent_down, latent_up, blob, k, F, bias=None, renormalize=True, act="bf16", down=None,
          up=None):
    """The layer on CPU tensors (blob: numpy records).  down / up: (stack, ids, rank) or None.
    Returns (out fp64 before its rounding, idx, w)."""
    T, E, L = x.shape[0], router_w.shape[0], latent_down.shape[0]
    logits = (x.double() @ router_w.double().T).float()
    if bias is not None:
        logits = logits + bias
    act_of = mxfp8 if act == "mxfp8" else (lambda v: v)
    h = act_of(round_bf16(linear(x, latent_down, *(down or ()))[0]))
    idx, w = torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k), dtype=torch.float64)
    z = torch.zeros((T, L), dtype=torch.float64)
    cache = {}
    for t in range(T):
        row = logits[t].tolist()
        best = sorted(sorted(range(E), key=lambda e: (-row[e], e))[:k])
        lt = logits[t].double()
        p = torch.softmax(lt[best], 0) if renormalize else torch.softmax(lt, 0)[best]
        for j, e in enumerate(best):
            if e not in cache:
                cache[e] = expert(blob, e, L, F)
            g, u = cache[e][0] @ h[t], cache[e][1] @ h[t]
            a = act_of(round_bf16(g / (1 + torch.exp(-g)) * u)[None])[0]
            z[t] += p[j] * (cache[e][2] @ a)
            idx[t, j], w[t, j] = e, p[j]
    return linear(round_bf16(z).bfloat16(), latent_up, *(up or ()))[0], idx, w
