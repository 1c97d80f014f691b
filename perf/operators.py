"""What is measured of the library's adapter and few-token operators, and their plain forms.

Three calls are covered:

 * ``linear_lora``: the shared bf16 projection of a batch with one low-rank adapter per
   request beside it (multi-tenant serving),
       u[t]   = A[a_t] x[t]                                  (fp32, a_t the token's adapter)
       out[t] = bf16(W x[t] + scale[a_t] B[a_t] u[t])        (a_t = -1: W x[t] alone);
 * ``layer_decode``: the whole Stable-LatentMoE layer for the few tokens of a decode step,
   with adapters on the latent projections or without;
 * ``layer_lora``: the same layer with adapters through ``layer_forward`` (a larger batch).

The layer is the library's: router logits are the correctly rounded fp32 dot products plus the
bias, the top k (ties to the lower index) are weighted by a softmax over them, and its latent
row h, its GLU rows a and its combined row z are bf16 values by definition (MXFP8 mode: h and a
are quantised to MXFP8 after that), so every form rounds there:
       h = bf16(Wd x [+ adapter]), a = bf16(silu(Wg h) Wu h), z = bf16(sum_j w_j Wdn a_j),
       out = bf16(Wu z [+ adapter]).
"""
import math

import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------------------- cases

def _lora(name, tokens, n_in, n_out, adapters, max_rank, order, ragged, none):
    return dict(name=name, op="linear_lora", tokens=tokens, n_in=n_in, n_out=n_out, adapters=adapters,
                max_rank=max_rank, order=order, ragged=ragged, none=none)


def _layer(name, op, tokens, d, L, F, E, k, layout, act="bf16", bias="none", adapters=0, max_rank=0):
    return dict(name=name, op=op, tokens=tokens, d_model=d, d_latent=L, d_ffn=F, experts=E, top_k=k, layout=layout,
                act=act, bias=bias, adapters=adapters, max_rank=max_rank)


K3 = (7168, 3584, 3072, 896, 16)  # the K3-shaped layer of the benchmark


def listed():
    return [
        # the smallest call: a tiny layer's down projection, where the launches are the cost
        _lora("lora_tiny", 16, 256, 128, 4, 8, "mixed", False, True),
        # one request decoding through the latent down projection, beside 31 idle adapters
        _lora("lora_one_token", 1, 7168, 3584, 32, 16, "mixed", False, False),
        # a decode batch of 64 requests, nearly each with an adapter of its own
        _lora("lora_decode64", 64, 7168, 3584, 64, 16, "mixed", False, True),
        # an odd decode batch on the up projection, few adapters of unequal ranks
        _lora("lora_batch33_up", 33, 3584, 7168, 9, 64, "mixed", True, True),
        # prompts of odd lengths, one after another, adapters of the largest rank
        _lora("lora_prompt1021_up", 1021, 3584, 7168, 5, 128, "segments", True, False),
        # a full prefill chunk of several requests' prompts
        _lora("lora_prefill4096", 4096, 7168, 3584, 16, 32, "segments", False, False),
        # a tiny layer decoding: five launches' worth of latency and little else
        _layer("decode_tiny", "layer_decode", 4, 256, 128, 128, 8, 2, "record"),
        # a mid-sized layer, MXFP8 activations, the widest batch of a decode step
        _layer("decode_mid_mxfp8", "layer_decode", 8, 2048, 1024, 512, 64, 8, "packed", act="mxfp8"),
        # one token through the benchmark's layer
        _layer("decode_k3_one", "layer_decode", 1, *K3, "packed"),
        # three tokens, checkpoint records as shipped, a router bias
        _layer("decode_k3_three", "layer_decode", 3, *K3, "record", bias="expert"),
        # two requests decoding, each with its adapter on both latent projections
        _layer("decode_k3_lora", "layer_decode", 2, *K3, "packed", adapters=8, max_rank=16),
        # a decode batch with adapters through the batch path
        _layer("layer_lora48", "layer_lora", 48, 1024, 512, 512, 64, 4, "packed", adapters=8, max_rank=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        tokens = _log_int(rng, 1, 4096)
        n_in = 32 * _log_int(rng, 4, 224)
        n_out = _log_int(rng, 64, 7168)
        while tokens * n_in * n_out > 4096 * 7168 * 3584:
            n_out = max(64, n_out // 2)
        max_rank = rng.choice([8, 16, 24, 32, 48, 64, 128])
        adapters = _log_int(rng, 1, 2048 // max(max_rank, 32))
        c = _lora("", tokens, n_in, n_out, adapters, max_rank, rng.choice(["mixed", "segments"]),
                  rng.random() < 0.5, rng.random() < 0.5)
    else:
        d, L, F = 128 * _log_int(rng, 1, 40), 128 * _log_int(rng, 1, 20), 128 * _log_int(rng, 1, 20)
        E = _log_int(rng, 4, 512)
        while E * 3 * L * F > 6_000_000_000:
            E //= 2
        k = rng.randint(1, min(E, 16))
        lora = rng.random() < 0.5
        op = "layer_lora" if lora and rng.random() < 0.4 else "layer_decode"
        tokens = _log_int(rng, 1, 32) if op == "layer_lora" else rng.randint(1, 8)
        while tokens * k > 64:
            k -= 1
        while tokens * k * L * F > 64 * 3584 * 1536:
            F = max(128, F - 128)
        c = _layer("", op, tokens, d, L, F, E, k, rng.choice(["packed", "record"]),
                   act=rng.choice(["bf16", "bf16", "mxfp8"]), bias=rng.choice(["none", "expert", "token"]),
                   adapters=rng.randint(1, 16) if lora else 0, max_rank=rng.choice([8, 16, 40, 64]) if lora else 0)
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs

def _normal(g, shape, std):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _adapters(g, c, n_in, n_out, tokens, order, ragged, none):
    """Adapters as a server holds them (one stack for all tenants) and the tokens' adapter ids."""
    N, R = c["adapters"], c["max_rank"]
    a = _normal(g, (N, R, n_in), n_in ** -0.5)
    b = _normal(g, (N, n_out, R), 0.05)
    scale = 0.5 + 2.0 * torch.rand(N, generator=g, device="cuda")
    rank = torch.randint(1, R + 1, (N,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    ids = torch.randint(-1 if none else 0, N, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    if order == "segments":  # whole prompts one after another
        cuts = torch.rand(tokens, generator=g, device="cuda") < 8.0 / max(tokens, 1)
        ids = ids[torch.cumsum(cuts, 0).clamp_max(tokens - 1)]
    return dict(a=a, b=b, scale=scale, rank=rank, adapter=ids.contiguous())


def _matrix_bytes(R, K, layout):
    return R * K // 2 + R * K // 32 if layout == "record" else R // 16 * (K // 128 * 1024 + (K // 128 + 3) // 4 * 256)


def _expert_bytes(c):
    L, F = c["d_latent"], c["d_ffn"]
    return 2 * _matrix_bytes(F, L, c["layout"]) + _matrix_bytes(L, F, c["layout"])


def _blob(g, c):
    """Experts as the checkpoint or the packed layout holds them: codes, then scales about 2^-8."""
    L, F, E, layout = c["d_latent"], c["d_ffn"], c["experts"], c["layout"]
    per = _expert_bytes(c)
    words = torch.randint(-2 ** 63, 2 ** 63 - 1, ((E * per + 7) // 8,), generator=g, device="cuda", dtype=torch.int64)
    blob = words.view(torch.uint8)[: E * per]
    at, e = 0, blob.view(E, per)
    for R, K in ((F, L), (F, L), (L, F)):
        m = e[:, at: at + _matrix_bytes(R, K, layout)]
        s = m[:, R * K // 2:] if layout == "record" else m.unflatten(1, (R // 16, -1))[:, :, K // 128 * 1024:]
        s.copy_(torch.randint(118, 121, s.shape, generator=g, device="cuda", dtype=torch.uint8))
        at += _matrix_bytes(R, K, layout)
    return blob


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, T = case, case["tokens"]
    if c["op"] == "linear_lora":
        s = dict(x=_normal(g, (T, c["n_in"]), 1.0), W=_normal(g, (c["n_out"], c["n_in"]), 0.02),
                 lora=_adapters(g, c, c["n_in"], c["n_out"], T, c["order"], c["ragged"], c["none"]))
    else:
        d, L, E = c["d_model"], c["d_latent"], c["experts"]
        s = dict(x=_normal(g, (T, d), 1.0), router_w=_normal(g, (E, d), 0.02), latent_down=_normal(g, (L, d), 0.02),
                 latent_up=_normal(g, (d, L), 0.02), blob=_blob(g, c), bias=None, down=None, up=None)
        if c["bias"] != "none":
            s["bias"] = torch.randn((E,) if c["bias"] == "expert" else (T, E), generator=g, device="cuda")
        if c["adapters"]:
            s["down"] = _adapters(g, c, d, L, T, "mixed", True, T > 4)
            s["up"] = _adapters(g, c, L, d, T, "mixed", True, T > 4)
            s["up"]["adapter"] = s["down"]["adapter"]  # a request's adapter covers both projections
    s["case"] = c
    return s


# --------------------------------------------------------------------------- plain forms

def _plain_linear(x, W, lo=None):
    """W x and the adapters' term in fp32: the products with every adapter at once, of which a
    mask keeps the token's own."""
    out = x.float() @ W.float().T
    if lo is None:
        return out
    N, R, n_in = lo["a"].shape
    at = torch.arange(N, device=x.device, dtype=torch.int32)
    live = (lo["adapter"][:, None] == at)[:, :, None].expand(-1, -1, R)
    if lo["rank"] is not None:
        live = live & (torch.arange(R, device=x.device) < lo["rank"][:, None])
    u = (x.float() @ lo["a"].view(N * R, n_in).float().T).view(-1, N, R) * lo["scale"][:, None]
    u = torch.where(live, u, torch.zeros_like(u)).view(-1, N * R)
    return out + u @ lo["b"].float().transpose(1, 2).reshape(N * R, -1)


def _plain_matrices(c, blob, ids):
    """fp32 gate [n, F, L], up [n, F, L] and down [n, L, F] of the experts `ids`."""
    L, F, E, layout = c["d_latent"], c["d_ffn"], c["experts"], c["layout"]
    half = torch.tensor(E2M1 + [-v for v in E2M1], device=blob.device)
    pair = torch.stack((half.repeat(16), half.repeat_interleave(16)), 1)  # byte -> (low nibble, high nibble)
    rec = blob.view(E, -1)[ids]
    n, at, found = len(ids), 0, []
    for R, K in ((F, L), (F, L), (L, F)):
        m = rec[:, at: at + _matrix_bytes(R, K, layout)]
        at += _matrix_bytes(R, K, layout)
        if layout == "record":
            codes, scales = m[:, : R * K // 2], m[:, R * K // 2:]
        else:  # 16-row groups of [step][block][row][16 bytes], then of [4 steps][block][row][step]
            grp, nks = m.unflatten(1, (R // 16, -1)), K // 128
            codes = grp[:, :, : nks * 1024].unflatten(2, (nks, 4, 16, 16)).permute(0, 1, 4, 2, 3, 5)
            scales = grp[:, :, nks * 1024:].unflatten(2, (-1, 4, 16, 4)).permute(0, 1, 4, 2, 5, 3)
            scales = scales.reshape(n, R, -1)[:, :, : K // 32]
        w = pair[codes.reshape(n, R, K // 2).int()].view(n, R, K // 32, 32)
        found.append((w * _pow2(scales.reshape(n, R, K // 32, 1).int() - 127)).view(n, R, K))
    return found


def _bf16(v):
    return v.bfloat16().float()


def _pow2(e):
    """2^e of whole e in [-126, 127], exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_mxfp8(v):
    """The values that MXFP8 holds of rows v: blocks of 32 with scale 2^(floor(log2 max) - 8)."""
    blk = v.unflatten(-1, (-1, 32))
    top = blk.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 9).clamp(-126, 126)
    q = (blk * _pow2(-e)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * _pow2(e)).flatten(-2)


def _plain_layer(s):
    c, x = s["case"], s["x"]
    T, k = c["tokens"], c["top_k"]
    act = _plain_mxfp8 if c["act"] == "mxfp8" else (lambda v: v)
    logits = (x.double() @ s["router_w"].double().T).float()  # a border between two experts needs more than 32 bits
    if s["bias"] is not None:
        logits = logits + s["bias"]
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k].sort(dim=1)[0]
    w = torch.softmax(logits.gather(1, idx), dim=1)
    h = act(_bf16(_plain_linear(x, s["latent_down"], s["down"])))
    gate, up, down = _plain_matrices(c, s["blob"], idx.flatten())
    rows = h.repeat_interleave(k, 0)[:, :, None]
    g, u = torch.bmm(gate, rows)[:, :, 0], torch.bmm(up, rows)[:, :, 0]
    a = act(_bf16(g / (1.0 + torch.exp(-g)) * u))
    y = torch.bmm(down, a[:, :, None])[:, :, 0]
    z = (w[:, :, None] * y.view(T, k, -1)).sum(1).bfloat16()
    out = _plain_linear(z, s["latent_up"], s["up"]).bfloat16()
    return dict(out=out, topk_idx=idx.int(), topk_w=w)


# ---------------------------------------------------------------------- the library's calls

def _own_lora(moe, lo):
    return None if lo is None else moe.Lora(lo["a"], lo["b"], lo["scale"], lo["adapter"], lo["rank"])


def _own(s):
    import mxfp4_expert_gemm_amd as moe

    c, x = s["case"], s["x"]
    if c["op"] == "linear_lora":
        return moe.linear_lora(x, s["W"], _own_lora(moe, s["lora"]))
    T, k = c["tokens"], c["top_k"]
    routing = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device=x.device),
                   topk_w=torch.empty((T, k), dtype=torch.float32, device=x.device))
    call = moe.layer_decode if c["op"] == "layer_decode" else moe.layer_forward
    out = call(x, s["router_w"], s["latent_down"], s["latent_up"], s["blob"], k, d_ffn=c["d_ffn"], bias=s["bias"],
               routing=routing, packed=c["layout"] == "packed",
               act_format=moe.ACT_FMT_MXFP8 if c["act"] == "mxfp8" else moe.ACT_FMT_BF16,
               lora_down=_own_lora(moe, s["down"]), lora_up=_own_lora(moe, s["up"]))
    return dict(out=out, **routing)


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "linear_lora":
        return _plain_linear(state["x"], state["W"], state["lora"]).bfloat16()
    return _plain_layer(state)


# ---------------------------------------------------------------------------------- work

def _distinct(n, draws):
    """How many of n are met in so many independent draws."""
    return n * (1.0 - (1.0 - 1.0 / n) ** draws)


def _lora_work(T, n_in, n_out, N, R):
    return _distinct(N, T) * R * (n_in + n_out) * 2, 2 * T * R * (n_in + n_out)


def work(case):
    c, T = case, case["tokens"]
    if c["op"] == "linear_lora":
        n_in, n_out = c["n_in"], c["n_out"]
        met = T if c["order"] == "mixed" else min(T, 9)
        lb, lf = _lora_work(met, n_in, n_out, c["adapters"], c["max_rank"])
        return dict(bytes=2 * (T * n_in + n_in * n_out + T * n_out) + lb,
                    flops=2 * T * n_in * n_out + lf * T / met)
    d, L, F, E, k = (c[n] for n in ("d_model", "d_latent", "d_ffn", "experts", "top_k"))
    active = E * (1.0 - (1.0 - k / E) ** T)
    b = 2 * (E * d + 2 * d * L + 2 * T * d) + active * _expert_bytes(c) + 8 * T * k
    f = 2 * T * (E * d + 2 * d * L + 3 * k * L * F)
    if c["adapters"]:
        lb, lf = _lora_work(T, d, L, c["adapters"], c["max_rank"])
        b, f = b + 2 * lb, f + 2 * lf
    return dict(bytes=b, flops=f)


# --------------------------------------------------------------------------------- exact

def _exact_linear(x, W, lo):
    """Row by row of the definition, in fp64, each adapter on the tokens that name it."""
    x = x.double()
    out = torch.matmul(x, W.double().t())
    if lo is not None:
        for i in sorted(set(lo["adapter"].tolist()) - {-1}):
            r = lo["a"].shape[1] if lo["rank"] is None else int(lo["rank"][i])
            rows = (lo["adapter"] == i).nonzero()[:, 0]
            u = torch.matmul(x[rows], lo["a"][i, :r].double().t())
            out[rows] += float(lo["scale"][i]) * torch.matmul(u, lo["b"][i, :, :r].double().t())
    return out


def _two(e):
    """2^e of whole e in fp64, exactly (the device's pow is an ulp off at some of them)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_weight(c, blob, e, which):
    """Matrix `which` (0 gate, 1 up, 2 down) of expert e in fp64, each weight found at its own place."""
    L, F, layout = c["d_latent"], c["d_ffn"], c["layout"]
    R, K = (L, F) if which == 2 else (F, L)
    base = e * _expert_bytes(c) + which * _matrix_bytes(F, L, layout)
    row = torch.arange(R, device=blob.device)[:, None]
    byte, blk = torch.arange(K // 2, device=blob.device), torch.arange(K // 32, device=blob.device)
    if layout == "record":
        at_code, at_scale = row * (K // 2) + byte, R * K // 2 + row * (K // 32) + blk
    else:
        nks = K // 128
        start = row // 16 * (nks * 1024 + (nks + 3) // 4 * 256)
        at_code = start + byte // 64 * 1024 + 16 * (row % 16 + 16 * (byte % 64 // 16)) + byte % 16
        step = blk // 4
        at_scale = start + nks * 1024 + step // 4 * 256 + 4 * (row % 16 + 16 * (blk % 4)) + step % 4
    code = blob[base + at_code].long()
    code = torch.stack((code & 15, code >> 4), -1).view(R, K)
    ex, man = code >> 1 & 3, (code & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * _two(ex - 1))
    val = torch.where(code >= 8, -mag, mag)
    return val * _two(blob[base + at_scale].long() - 127).repeat_interleave(32, 1)


def _exact_round(v, bits, low):
    """v to the nearest value of `bits` significant bits, ties to even, steps no finer than 2^low."""
    step = _two((torch.frexp(v)[1] - bits).clamp(min=low))
    return torch.round(v / step) * step


def _exact_act(c, v):
    v = _exact_round(v, 8, -133)
    if c["act"] != "mxfp8":
        return v
    b = v.view(-1, v.shape[-1] // 32, 32)
    top = b.abs().max(-1, keepdim=True)[0]
    x = _two((torch.frexp(top)[1] - 1 - 8).clamp(min=-127))
    return (_exact_round(b / x, 4, -9).clamp(-448.0, 448.0) * x).view_as(v)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "linear_lora":
        return _exact_linear(s["x"], s["W"], s["lora"])
    k = c["top_k"]
    logits = torch.matmul(s["x"].double(), s["router_w"].double().t()).float()
    logits = logits if s["bias"] is None else logits + s["bias"]
    h = _exact_act(c, _exact_linear(s["x"], s["latent_down"], s["down"]))
    idx = torch.empty((c["tokens"], k), dtype=torch.int32, device=h.device)
    w = torch.empty((c["tokens"], k), dtype=torch.float64, device=h.device)
    z = torch.zeros((c["tokens"], c["d_latent"]), dtype=torch.float64, device=h.device)
    for t, row in enumerate(logits.tolist()):
        best = sorted(sorted(range(len(row)), key=lambda e: (-row[e], e))[:k])
        p = [math.exp(row[e] - max(row)) for e in best]
        for j, e in enumerate(best):
            idx[t, j], w[t, j] = e, p[j] / math.fsum(p)
            g, u = _exact_weight(c, s["blob"], e, 0) @ h[t], _exact_weight(c, s["blob"], e, 1) @ h[t]
            a = _exact_act(c, (g * torch.sigmoid(g) * u)[None])[0]
            z[t] += w[t, j] * (_exact_weight(c, s["blob"], e, 2) @ a)
    return dict(out=_exact_linear(_exact_round(z, 8, -133), s["latent_up"], s["up"]), topk_idx=idx, topk_w=w)
