"""The dense block, the norms between blocks and the 8-bit projection run together: a residual stream
over a stack of dense and routed layers down to a projection, and a training step through blocks."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import plain_ffn
import plain_int8
import plain_norms
import synth
from gpu_common import to_dev
from mxfp4_expert_gemm_amd.stream import LayerStack

pytestmark = pytest.mark.gpu

EPS = moe.NORM_EPS


def b(shape, std, seed, mean=0.0):
    return (mean + plain.bf16(shape, std, seed)).cuda()


def dense_layer(d, F, seed, T=None):
    """a gated block with all that may stand around it; T: its gate is one row a token"""
    return dict(w_gate=b((F, d), d ** -0.5, seed), w_up=b((F, d), d ** -0.5, seed + 1),
                w_down=b((d, F), F ** -0.5, seed + 2), pre_norm=b((d,), 0.2, seed + 3, 1.0),
                post_norm=b((d,), 0.2, seed + 4, 1.0), gate=b((d,) if T is None else (T, d), 1.0, seed + 5), scale=0.75)


def routed_layer(c, seed):
    d, L = c.d, c.L
    return dict(router_w=to_dev(synth.normal_bf16(seed, 2, 0.02, (c.E, d))).view(torch.bfloat16),
                latent_down=to_dev(synth.normal_bf16(seed, 3, 0.02, (L, d))).view(torch.bfloat16),
                latent_up=to_dev(synth.normal_bf16(seed, 4, 0.02, (d, L))).view(torch.bfloat16),
                expert_blob_host=torch.from_numpy(synth.expert_blob(seed, L, c.F, c.E)).pin_memory())


def check(got, want, what):
    for name, (v, bound) in want.items():
        t = got[name]
        assert torch.isfinite(t).all(), (what, name)
        off = (t.double() - v).abs() - bound
        assert off.max() <= 0, (what, name, off.max().item())


def by_hand(stack, x, final, head=None):
    """The stack's pass by single calls with tensors of their own; [(layer, its input, result, stream)] too."""
    residual, seen = x, []
    for i, lay in enumerate(stack.layers):
        n = residual
        if lay.get("pre_norm") is not None:
            n = moe.block_norms(None, residual, pre_weight=lay["pre_norm"])[1]
        y = torch.empty_like(x)
        stack.forward_layer(i, n, out=y)
        after = moe.block_norms(y, residual, post_weight=lay.get("post_norm"), gate=lay.get("gate"),
                                scale=lay.get("scale", 1.0))[0]
        seen.append((lay, residual, n, y, after))
        residual = after
    n = moe.block_norms(None, residual, pre_weight=final)[1]
    return residual, n, seen


@pytest.mark.parametrize("T", [1, 5, 33, 300])
def test_dense_stack(T):
    """Every tensor on the way against the plain forms, and the pass against single calls bit for bit."""
    d = 512
    layers = [dense_layer(d, 344, 10), dense_layer(d, 1000, 20, T), dense_layer(d, 512, 30)]
    layers[2].update(pre_norm=None, gate=None)
    stack = LayerStack(layers, 0, 0, 0, T)
    x, final = b((T, d), 1.0, 1), b((d,), 0.2, 2, 1.0)
    keep = x.clone()
    residual, n, seen = by_hand(stack, x, final)
    for i, (lay, before, h, y, after) in enumerate(seen):
        if lay["pre_norm"] is not None:
            check(dict(normed=h), plain_norms.forward(None, before, lay["pre_norm"], None, None, 1.0, EPS, before), i)
        check(dict(out=y), dict(out=plain_ffn.forward(h, lay["w_gate"], lay["w_up"], lay["w_down"])["out"]), i)
        check(dict(out=after), plain_norms.forward(y, before, None, lay["post_norm"], lay["gate"], lay["scale"], EPS,
                                                   after), i)
    W, ws = moe.quantize_int8(b((1000, d), d ** -0.5, 3))
    got = stack.forward(x, final_norm=final, head=(W, ws))
    assert torch.equal(x, keep) and torch.equal(got[0], residual)
    q, qs = plain_int8.codes(n.cpu())
    logits = plain_int8.product(q, torch.from_numpy(qs), W.cpu(), ws.cpu())
    # exact sums, two fp32 products and the rounding
    assert ((got[1].cpu().double() - logits).abs() <= logits.abs() * (2.0 ** -8 + 2.0 ** -21)).all()
    assert torch.equal(stack.forward(x, final_norm=final)[1], n)
    last = stack.forward(x)
    assert torch.equal(last[0], residual) and last[1] is None
    wide = W.bfloat16()
    assert torch.equal(stack.forward(x, final_norm=final, head=wide)[1], moe.linear_bf16(n, wide))


@pytest.mark.parametrize("T", [1, 40])
def test_dense_and_routed_layers(T):
    """A dense layer before routed ones, as the model has it, and behind; where the experts live changes nothing."""
    c = synth.CONFIGS["tiny"]
    d = c.d
    layers = [dense_layer(d, 256, 10), routed_layer(c, 0x51), dict(routed_layer(c, 0x52), pre_norm=b((d,), 0.2, 4, 1.0)),
              dense_layer(d, 344, 20), dict(routed_layer(c, 0x53), gate=b((d,), 1.0, 5), scale=2.0)]
    x, final = b((T, d), 1.0, 1), b((d,), 0.2, 2, 1.0)
    head = moe.quantize_int8(b((256, d), d ** -0.5, 3))
    want = None
    for pinned in (5, 2, 0):
        stack = LayerStack(layers, c.k, c.F, pinned, T)
        assert (stack.slots is None) == (pinned == 5)
        residual, n, _ = by_hand(stack, x, final)
        got = stack.forward(x, final_norm=final, head=head)
        assert torch.isfinite(got[0].float()).all()
        assert torch.equal(got[0], residual) and torch.equal(got[1], moe.linear_int8(n, *head))
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 20])
def test_captured_pass_and_side_stream(T):
    """A pass over resident layers captured into a graph and replayed on new contents, with eager work
    between the replays, and one given a stream of its own: the eager pass's bits."""
    c = synth.CONFIGS["tiny"]
    d = c.d
    stack = LayerStack([dense_layer(d, 344, 10), routed_layer(c, 0x51), dense_layer(d, 256, 20)], c.k, c.F, 3, T)
    x, final = b((T, d), 1.0, 1), b((d,), 0.2, 2, 1.0)
    kw = dict(final_norm=final, head=moe.quantize_int8(b((256, d), d ** -0.5, 3)))
    stack.forward(x, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res, logits = stack.forward(x, **kw)
    for seed in (5, 6, 7):
        x.copy_(plain.bf16((T, d), 1.0, seed))
        want = stack.forward(x, **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = stack.forward(x, stream=side, **kw)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        res.fill_(float("nan"))
        logits.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, want[0]) and torch.equal(logits, want[1])


class Round(torch.autograd.Function):
    """bf16 where the kernels round: the value, its gradient, or both"""

    @staticmethod
    def forward(ctx, v, value, grad):
        ctx.grad = grad
        return v.bfloat16().double() if value else v.clone()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double() if ctx.grad else g, None, None


def chain(x, layers, final, rounded):
    """The residual stream over dense blocks in fp64 with autograd, with or without the roundings."""
    r = (lambda v, value=True, grad=True: Round.apply(v, value, grad)) if rounded else lambda v, *_: v
    norm = lambda v: plain_norms.norm(v, EPS)[0]
    for w in layers:
        h = r(norm(x) * w["pre_norm"])
        g, u = r(h @ w["w_gate"].T, False), r(h @ w["w_up"].T, False)
        a = r(g * plain_ffn.sigmoid(g) * u, True, False)
        y = r(a @ w["w_down"].T)
        x = r(x + w["scale"] * w["gate"] * norm(y) * w["post_norm"])
    return r(norm(x) * final, True, False)


@pytest.mark.parametrize("T,d,F", [(24, 256, 344), (300, 512, 1000)])
def test_training_step(T, d, F):
    """Two residual blocks forward and back by the calls, against autograd in fp64.

    The roundings to bf16 on the way are the whole error: fp32 sums are some 2^12 finer.  The fp64
    chain with roundings makes those but of the kept gate and up and of a token's gate gradient, one of
    six or more on each path, so its distance from the exact chain is at least sqrt(5/6) of what
    independent roundings give; the call's, of other such roundings, may be twice that, which leaves
    nearly half of it for their correlation."""
    layers = [dense_layer(d, F, 10), dense_layer(d, F, 20, T)]
    final, x, dn = b((d,), 0.2, 2, 1.0), b((T, d), 1.0, 1), b((T, d), 0.05, 3)

    # forward, keeping what the backward pass reads
    kept, residual, y, prev = [], x, None, {}
    for w in layers:
        residual, h = moe.block_norms(y, residual, pre_weight=w["pre_norm"], post_weight=prev.get("post_norm"),
                                      gate=prev.get("gate"), scale=prev.get("scale", 1.0))
        gate, up = (torch.empty(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        before = y
        y = moe.gated_ffn(h, w["w_gate"], w["w_up"], w["w_down"], gate=gate, up=up)
        kept.append((before, residual, h, gate, up))
        prev = w
    out, n = moe.block_norms(y, residual, pre_weight=final, post_weight=prev["post_norm"], gate=prev["gate"],
                             scale=prev["scale"])
    # and back
    got = {}
    s = moe.block_norms_backward(None, dn, y, out, post_weight=prev["post_norm"], pre_weight=final, gate=prev["gate"],
                                 scale=prev["scale"])
    got["final"] = s.dpre_weight
    for i in (1, 0):
        w, (before, res, h, gate, up) = layers[i], kept[i]
        got[f"post_norm{i}"], got[f"gate{i}"] = s.dpost_weight, s.dgate
        f = moe.gated_ffn_backward(s.dy, h, w["w_gate"], w["w_up"], w["w_down"], gate, up)
        got.update({f"w_gate{i}": f.dw_gate, f"w_up{i}": f.dw_up, f"w_down{i}": f.dw_down})
        p = layers[i - 1] if i else {}
        s = moe.block_norms_backward(s.dresidual, f.dx, before, res, post_weight=p.get("post_norm"),
                                     pre_weight=w["pre_norm"], gate=p.get("gate"), scale=p.get("scale", 1.0))
        got[f"pre_norm{i}"] = s.dpre_weight
    got["x"] = s.dresidual

    def plain_grads(rounded):
        leaf = lambda t: t.cpu().double().requires_grad_()
        ls = [{k: v if k == "scale" else leaf(v) for k, v in w.items()} for w in layers]
        xs, fs = leaf(x), leaf(final)
        v = chain(xs, ls, fs, rounded)
        v.backward(dn.cpu().double())
        g = {f"{k}{i}": t.grad for i, w in enumerate(ls) for k, t in w.items() if k != "scale"}
        return v.detach(), {**g, "x": xs.grad, "final": fs.grad}

    (exact, ge), (near, gr) = plain_grads(False), plain_grads(True)
    ge["n"], gr["n"], got["n"] = exact, near, n
    assert set(ge) == set(got)
    for name, e in ge.items():
        t = got[name].cpu().double()
        assert t.shape == e.shape, name
        limit = 2 * (gr[name] - e).norm()
        assert (t - e).norm() <= limit, (name, ((t - e).norm() / e.norm()).item(), (limit / e.norm()).item())
    # along a direction of each input the plain chain changes as its gradient says, by differences
    for name, t in (("x", x), ("final", final), ("w_down1", layers[1]["w_down"]), ("gate0", layers[0]["gate"])):
        way = torch.randn(t.shape, generator=torch.Generator().manual_seed(7), dtype=torch.float64)
        step, at = 1e-5, {}
        for sign in (1, -1):
            ls = [{k: v if k == "scale" else v.cpu().double() for k, v in w.items()} for w in layers]
            xs, fs = x.cpu().double(), final.cpu().double()
            place = {"x": xs, "final": fs, "w_down1": ls[1]["w_down"], "gate0": ls[0]["gate"]}[name]
            place += sign * step * way
            at[sign] = (chain(xs, ls, fs, False) * dn.cpu().double()).sum()
        slope = (at[1] - at[-1]) / (2 * step)
        # off by what the gradient is off, at most the limit above times the direction's length, and the
        # differences' own error, 1e-6 of the terms' sizes and more
        limit = 2 * (gr[name] - ge[name]).norm() * way.norm() + 1e-5 * ge[name].norm() * way.norm()
        assert ((got[name].cpu().double() * way).sum() - slope).abs() <= limit, name
