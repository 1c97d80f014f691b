"""What is measured of the library's dense block, block norms and 8-bit projection, and their plain forms.

Five calls are covered:

 * ``gated_ffn``: the dense gated feed-forward block,
       g = Wg x, u = Wu x, out = Wd (silu(g) u),
   for serving, and for training, where bf16(g) and bf16(u) are kept for its backward pass;
 * ``gated_ffn_backward``: the gradients of x and the three matrices from dout and the kept g, u;
 * ``block_norms``: what stands between two blocks of a residual stream,
       out    = bf16(residual + scale * gate * norm(y) * post_weight),
       normed = bf16(norm(out) * pre_weight),   norm(v) = v / sqrt(mean(v^2) + eps),
   with a gate per channel, one per token and channel, or none.  The second norm is that of the
   stored stream, so every form rounds out before it;
 * ``block_norms_backward``: the gradients of all of its inputs;
 * ``linear_int8``: a projection whose tokens are quantised to 8 bits on the way in,
       q = round(127 x / max|x|) per token, out = bf16(x_scale * w_scale * sum q W).
"""
import math

import torch

own = False

EPS = 2.0 ** -23


# ------------------------------------------------------------------------------- cases

def _ffn(name, op, tokens, d, F, save=False):
    return dict(name=name, op=op, tokens=tokens, d_model=d, d_ffn=F, save=save)


def _norms(name, op, tokens, d, gate, scale, post=True):
    return dict(name=name, op=op, tokens=tokens, d_model=d, gate=gate, scale=scale, post=post)


def _int8(name, tokens, n_in, n_out):
    return dict(name=name, op="linear_int8", tokens=tokens, n_in=n_in, n_out=n_out)


def listed():
    return [
        # a few tokens through a tiny block of odd widths: the launches are the cost
        _ffn("ffn_tiny", "gated_ffn", 5, 256, 344),
        # one token decoding through a dense layer of the benchmark's width
        _ffn("ffn_one_token", "gated_ffn", 1, 7168, 8192),
        # an odd decode batch through a block of the latent width
        _ffn("ffn_decode33", "gated_ffn", 33, 3584, 7168),
        # a training step's forward pass, g and u kept for the backward
        _ffn("ffn_train4096", "gated_ffn", 4096, 7168, 3584, save=True),
        # fine-tuning a small block on a short odd batch
        _ffn("ffn_back77", "gated_ffn_backward", 77, 512, 1000),
        # the backward pass of a training step
        _ffn("ffn_back4096", "gated_ffn_backward", 4096, 4096, 8192),
        # one token decoding: the stream between two layers
        _norms("norms_one_token", "block_norms", 1, 7168, "channel", 1.0),
        # a prefill chunk, each token's channels gated
        _norms("norms_prefill8192", "block_norms", 8192, 7168, "token", 0.5),
        # an odd small batch's backward, no norm after the block and no gate
        _norms("norms_back333", "block_norms_backward", 333, 1000, "none", 0.25, post=False),
        # a training step's backward with a learned gate of each channel
        _norms("norms_back8192", "block_norms_backward", 8192, 4096, "channel", 1.0),
        # a decode batch through the 8-bit latent down projection
        _int8("int8_decode48", 48, 7168, 3584),
        # a long odd prompt through the 8-bit latent up projection
        _int8("int8_prompt8191", 8191, 3584, 7168),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_ffn", "gated_ffn", "gated_ffn_backward", "block_norms", "block_norms_backward",
                     "linear_int8"])
    if op.startswith("gated_ffn"):
        tokens, d, F = _log_int(rng, 1, 4096), 8 * _log_int(rng, 8, 896), 8 * _log_int(rng, 8, 1024)
        while tokens * d * F > 100_000_000_000:
            tokens //= 2
        c = _ffn("", op, tokens, d, F, save=op == "gated_ffn" and rng.random() < 0.5)
    elif op.startswith("block_norms"):
        c = _norms("", op, _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 896),
                   rng.choice(["none", "channel", "token"]), rng.choice([1.0, 0.5, 0.125]), post=rng.random() < 0.7)
    else:
        c = _int8("", _log_int(rng, 1, 8192), 16 * _log_int(rng, 4, 512), _log_int(rng, 16, 8192))
        while c["tokens"] * c["n_in"] * c["n_out"] > 8191 * 3584 * 7168:
            c["tokens"] //= 2
    del c["name"]
    return c


# ------------------------------------------------------------------------------ inputs

def _normal(g, shape, std, mean=0.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(mean, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, T = case, case["tokens"]
    s = dict(case=c)
    if c["op"].startswith("gated_ffn"):
        d, F = c["d_model"], c["d_ffn"]
        s.update(x=_normal(g, (T, d), 1.0), w_gate=_normal(g, (F, d), d ** -0.5), w_up=_normal(g, (F, d), d ** -0.5),
                 w_down=_normal(g, (d, F), F ** -0.5))
        if c["op"] == "gated_ffn_backward":  # what the forward pass kept, and the gradient that comes back
            s["gate"] = (s["x"].float() @ s["w_gate"].float().T).bfloat16()
            s["up"] = (s["x"].float() @ s["w_up"].float().T).bfloat16()
            s["dout"] = _normal(g, (T, d), 0.01)
    elif c["op"].startswith("block_norms"):
        d = c["d_model"]
        s.update(y=_normal(g, (T, d), 3.0), pre_weight=_normal(g, (d,), 0.1, 1.0), post_weight=None, gate=None)
        if c["post"]:
            s["post_weight"] = _normal(g, (d,), 0.1, 1.0)
        if c["gate"] != "none":
            s["gate"] = _normal(g, (d,) if c["gate"] == "channel" else (T, d), 0.5, 0.5)
        stream = _normal(g, (T, d), 2.0)
        if c["op"] == "block_norms":
            s["residual"] = stream
        else:
            s.update(out=stream, dout=_normal(g, (T, d), 0.01), dnormed=_normal(g, (T, d), 0.01))
    else:
        s["x"] = _normal(g, (T, c["n_in"]), 1.0)
        w = _normal(g, (c["n_out"], c["n_in"]), 0.02).float()  # quantised once, when the weights are loaded
        top = w.abs().amax(1, keepdim=True)
        s["w_scale"] = (top / 127.0)[:, 0].contiguous()
        s["W"] = torch.round(w * 127.0 / top).to(torch.int8)
    return s


# --------------------------------------------------------------------------- plain forms

def _plain_ffn(s):
    g, u = s["x"].float() @ s["w_gate"].float().T, s["x"].float() @ s["w_up"].float().T
    out = (g / (1.0 + torch.exp(-g)) * u) @ s["w_down"].float().T
    found = dict(out=out.bfloat16())
    if s["case"]["save"]:
        found.update(gate=g.bfloat16(), up=u.bfloat16())
    return found


def _plain_ffn_backward(s):
    x, dout, g, u = s["x"].float(), s["dout"].float(), s["gate"].float(), s["up"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    da = dout @ s["w_down"].float()
    dg, du = da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig
    return dict(dx=(dg @ s["w_gate"].float() + du @ s["w_up"].float()).bfloat16(), dw_gate=(dg.T @ x).bfloat16(),
                dw_up=(du.T @ x).bfloat16(), dw_down=(dout.T @ (g * sig * u)).bfloat16())


def _inverse_rms(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _plain_norms(s):
    y = s["y"].float()
    if s["post_weight"] is not None:
        y = y * _inverse_rms(y) * s["post_weight"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    out = (s["residual"].float() + s["case"]["scale"] * y).bfloat16()
    v = out.float()
    return dict(out=out, normed=(v * _inverse_rms(v) * s["pre_weight"].float()).bfloat16())


def _plain_norms_backward(s):
    scale, r, dn = s["case"]["scale"], s["out"].float(), s["dnormed"].float()
    ir = _inverse_rms(r)
    rh, e = r * ir, dn * s["pre_weight"].float()
    d = s["dout"].float() + ir * (e - rh * (e * rh).mean(1, keepdim=True))
    found = dict(dresidual=d.bfloat16(), dpre_weight=(dn * rh).sum(0))
    y = s["y"].float()
    ih = _inverse_rms(y)
    yh = y * ih
    v, dv = y, scale * d
    if s["post_weight"] is not None:
        v = yh * s["post_weight"].float()
    if s["gate"] is not None:
        found["dgate"] = (dv * v).sum(0) if s["gate"].dim() == 1 else (dv * v).bfloat16()
        dv = dv * s["gate"].float()
    if s["post_weight"] is not None:
        found["dpost_weight"] = (dv * yh).sum(0)
        f = dv * s["post_weight"].float()
        dv = ih * (f - yh * (f * yh).mean(1, keepdim=True))
    found["dy"] = dv.bfloat16()
    return found


def _plain_int8(s):
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127.0 / top)  # 127 x is exact, its quotient is never rounded onto a border
    sums = (q.double() @ s["W"].double().T).float()  # whole sums past 2^24
    return (sums * (top / 127.0) * s["w_scale"]).bfloat16()


# ---------------------------------------------------------------------- the library's calls

def _own(s):
    import mxfp4_expert_gemm_amd as moe

    c = s["case"]
    if c["op"] == "gated_ffn":
        x = s["x"]
        kept = {}
        if c["save"]:
            kept = dict(gate=torch.empty((c["tokens"], c["d_ffn"]), dtype=x.dtype, device=x.device),
                        up=torch.empty((c["tokens"], c["d_ffn"]), dtype=x.dtype, device=x.device))
        return dict(out=moe.gated_ffn(x, s["w_gate"], s["w_up"], s["w_down"], **kept), **kept)
    if c["op"] == "gated_ffn_backward":
        return moe.gated_ffn_backward(s["dout"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"])._asdict()
    if c["op"] == "block_norms":
        out, normed = moe.block_norms(s["y"], s["residual"], pre_weight=s["pre_weight"], post_weight=s["post_weight"],
                                      gate=s["gate"], scale=c["scale"], eps=EPS)
        return dict(out=out, normed=normed)
    if c["op"] == "block_norms_backward":
        found = moe.block_norms_backward(s["dout"], s["dnormed"], s["y"], s["out"], pre_weight=s["pre_weight"],
                                         post_weight=s["post_weight"], gate=s["gate"], scale=c["scale"], eps=EPS)
        return found._asdict()
    return moe.linear_int8(s["x"], s["W"], s["w_scale"])


def run(state):
    if own:
        return _own(state)
    plain = dict(gated_ffn=_plain_ffn, gated_ffn_backward=_plain_ffn_backward, block_norms=_plain_norms,
                 block_norms_backward=_plain_norms_backward, linear_int8=_plain_int8)
    return plain[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------- work

def work(case):
    c, T = case, case["tokens"]
    if c["op"].startswith("gated_ffn"):
        d, F = c["d_model"], c["d_ffn"]
        if c["op"] == "gated_ffn":
            return dict(bytes=2 * (3 * d * F + 2 * T * d + (2 * T * F if c["save"] else 0)), flops=6 * T * d * F)
        return dict(bytes=2 * (6 * d * F + 3 * T * d + 2 * T * F), flops=12 * T * d * F)
    if c["op"].startswith("block_norms"):
        d, back = c["d_model"], c["op"] == "block_norms_backward"
        gate = dict(none=0, channel=2 * d, token=2 * T * d)[c["gate"]]
        weights = (2 + 4 * back) * d * (1 + c["post"])
        if c["gate"] == "channel" and back:
            weights += 4 * d
        if c["gate"] == "token" and back:
            gate *= 2
        return dict(bytes=2 * T * d * (6 if back else 4) + gate + weights, flops=T * d * (30 if back else 10))
    n, m = c["n_in"], c["n_out"]
    return dict(bytes=2 * T * n + n * m + 4 * m + 2 * T * m, flops=2 * T * n * m)


# --------------------------------------------------------------------------------- exact

def _exact_bf16(v):
    """v to the nearest value of 8 significant bits, ties to even."""
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v)[1] - 8)
    return torch.round(v / step) * step


def _exact_ffn(s):
    x = s["x"].double()
    g, u = torch.matmul(x, s["w_gate"].double().t()), torch.matmul(x, s["w_up"].double().t())
    out = torch.matmul(g * torch.sigmoid(g) * u, s["w_down"].double().t())
    return dict(out=out, gate=g, up=u) if s["case"]["save"] else dict(out=out)


def _exact_ffn_backward(s):
    """By the chain rule of log silu: d silu = silu (1/g + 1 - sigmoid), the quotient taken out."""
    g, u = s["gate"].double(), s["up"].double()
    p = torch.sigmoid(g)
    up = torch.matmul(s["dout"].double(), s["w_down"].double())
    back_u = up * (g * p)
    back_g = up * u * (p + g * p * torch.sigmoid(-g))
    x = s["x"].double()
    dx = torch.matmul(back_g, s["w_gate"].double())
    dx += torch.matmul(back_u, s["w_up"].double())
    return dict(dx=dx, dw_gate=torch.matmul(back_g.t(), x), dw_up=torch.matmul(back_u.t(), x),
                dw_down=torch.matmul(s["dout"].double().t(), g * p * u))


def _exact_norm(v):
    """v over its root mean square, and the matrix-free product with that map's transposed Jacobian."""
    n = v.shape[1]
    rms = (torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / n + EPS) ** 0.5
    unit = v / rms
    return unit, lambda t: (t - unit * torch.sum(t * unit, 1, keepdim=True) / n) / rms


def _exact_norms(s):
    c, y = s["case"], s["y"].double()
    if c["post"]:
        y = _exact_norm(y)[0] * s["post_weight"].double()
    gate = 1.0 if c["gate"] == "none" else s["gate"].double()
    out = s["residual"].double() + c["scale"] * (gate * y)
    return dict(out=out, normed=_exact_norm(_exact_bf16(out))[0] * s["pre_weight"].double())


def _exact_norms_backward(s):
    c, dn = s["case"], s["dnormed"].double()
    unit, back = _exact_norm(s["out"].double())
    stream = s["dout"].double() + back(dn * s["pre_weight"].double())
    found = dict(dresidual=stream, dpre_weight=torch.sum(dn * unit, 0))
    y, back = _exact_norm(s["y"].double()) if c["post"] else (s["y"].double(), lambda t: t)
    w = s["post_weight"].double() if c["post"] else 1.0
    gate = 1.0 if c["gate"] == "none" else s["gate"].double()
    if c["gate"] != "none":
        each = c["scale"] * stream * (y * w)
        found["dgate"] = torch.sum(each, 0) if c["gate"] == "channel" else each
    if c["post"]:
        found["dpost_weight"] = torch.sum(c["scale"] * stream * gate * y, 0)
    found["dy"] = back(c["scale"] * stream * gate * w)
    return found


def _exact_int8(s):
    x = s["x"].double()
    top = torch.max(torch.abs(x), 1, keepdim=True)[0]
    t = x * 127.0  # the nearest whole number to t / top; on a border the even one
    low = torch.floor(t / top)
    twice = 2.0 * (t - low * top)  # exact: few bits each
    up = (twice > top) | ((twice == top) & (low % 2 != 0))
    q = low + up
    sums = torch.matmul(q, s["W"].double().t())
    return sums * (top / 127.0) * s["w_scale"].double()


def exact(case, seed):
    forms = dict(gated_ffn=_exact_ffn, gated_ffn_backward=_exact_ffn_backward, block_norms=_exact_norms,
                 block_norms_backward=_exact_norms_backward, linear_int8=_exact_int8)
    return forms[case["op"]](prepare(case, seed))
