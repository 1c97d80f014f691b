"""The step between two blocks and its gradients against fp64 forms and differences: widths of every
kernel form, odd ones, all options, streams, captured graphs, rows that must not touch each other."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import plain_norms

pytestmark = pytest.mark.gpu

EPS = moe.NORM_EPS


def inputs(T, d, post, gate, seed=1):
    b = lambda shape, std, s: plain.bf16(shape, std, seed + s).cuda()
    return dict(y=b((T, d), 3.0, 0), residual=b((T, d), 2.0, 1), pre=1 + b((d,), 0.2, 2),
                post=1 + b((d,), 0.2, 3) if post else None,
                gate=None if gate == "none" else b((d,) if gate == "channel" else (T, d), 1.0, 4),
                dout=b((T, d), 0.01, 5), dnormed=b((T, d), 0.02, 6))


def check(got, want, what):
    for name, (v, bound) in want.items():
        t = got[name]
        assert torch.isfinite(t).all(), (what, name)
        off = (t.double() - v).abs() - bound
        assert off.max() <= 0, (what, name, off.max().item(), (t.double() - v).abs().max().item())


def forward(s, scale, **kw):
    out, normed = moe.block_norms(s["y"], s["residual"], pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                                  scale=scale, eps=EPS, **kw)
    return dict(out=out, normed=normed)


def backward(s, out, scale, **kw):
    return moe.block_norms_backward(s["dout"], s["dnormed"], s["y"], out, pre_weight=s["pre"], post_weight=s["post"],
                                    gate=s["gate"], scale=scale, eps=EPS, **kw)


# tokens and widths: one chunk, one wave's last column, each step of the pieces a thread holds, the
# widest, more rows than the backward's blocks hold at once, odd row counts in a block
SIZES = [(1, 8), (1, 7168), (2, 64), (3, 512), (5, 520), (7, 1000), (8, 1024), (9, 1032), (3, 2048), (4, 2056),
         (5, 4096), (2, 4104), (3, 6152), (2, 8192), (333, 1000), (1021, 24), (2049, 512), (4100, 1032), (777, 2056),
         (1500, 4104), (600, 8192)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("post,gate", [(True, "channel"), (True, "none"), (False, "token"), (False, "none")])
def test_both_passes(T, d, post, gate):
    s, scale = inputs(T, d, post, gate, seed=T + d), 0.5
    got = forward(s, scale)
    check(got, plain_norms.forward(s["y"], s["residual"], s["pre"], s["post"], s["gate"], scale, EPS, got["out"]), (T, d))
    grads = backward(s, got["out"], scale)
    check(grads._asdict(), plain_norms.backward(s["dout"], s["dnormed"], s["y"], got["out"], s["pre"], s["post"], s["gate"],
                                                scale, EPS), (T, d, post, gate))


@pytest.mark.parametrize("T,d", [(3, 264), (40, 3000)])
def test_every_subset_of_inputs(T, d):
    """No norm before the next block, the norm alone, one of the two gradients missing."""
    s = inputs(T, d, True, "token")
    out, none = moe.block_norms(s["y"], s["residual"], post_weight=s["post"], gate=s["gate"])
    assert none is None and torch.equal(out, forward(s, 1.0)["out"])
    grads = moe.block_norms_backward(s["dout"], None, s["y"], None, post_weight=s["post"], gate=s["gate"])
    check(grads._asdict(), plain_norms.backward(s["dout"], None, s["y"], None, None, s["post"], s["gate"], 1.0, EPS), "last")
    assert grads.dpre_weight is None and torch.equal(grads.dresidual, s["dout"])
    same, normed = moe.block_norms(None, s["residual"], pre_weight=s["pre"])
    assert same is s["residual"]
    check(dict(normed=normed), plain_norms.forward(None, s["residual"], s["pre"], None, None, 1.0, EPS, s["residual"]), "first")
    for dout, dnormed in ((None, s["dnormed"]), (s["dout"], s["dnormed"]), (s["dout"], None)):
        grads = moe.block_norms_backward(dout, dnormed, None, s["residual"], pre_weight=s["pre"])
        check(grads._asdict(), plain_norms.backward(dout, dnormed, None, s["residual"], s["pre"], None, None, 1.0, EPS), "first")
        assert grads.dy is None and grads.dgate is None
        grads = moe.block_norms_backward(dout, dnormed, s["y"], out, pre_weight=s["pre"], gate=s["gate"])
        check(grads._asdict(), plain_norms.backward(dout, dnormed, s["y"], out, s["pre"], None, s["gate"], 1.0, EPS), "middle")


def test_in_place():
    s = inputs(33, 1000, True, "channel")
    want = forward(s, 0.5)
    stream = s["residual"].clone()
    out, normed = moe.block_norms(s["y"], stream, pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"], scale=0.5,
                                  out=stream)
    assert out is stream and torch.equal(stream, want["out"]) and torch.equal(normed, want["normed"])
    grads = backward(s, out, 0.5)
    d = s["dout"].clone()
    again = moe.block_norms_backward(d, s["dnormed"], s["y"], out, pre_weight=s["pre"], post_weight=s["post"],
                                     gate=s["gate"], scale=0.5, grads=moe.BlockNormsGrads(d, None, None, None, None))
    assert again.dresidual is d and all(torch.equal(a, b) for a, b in zip(grads, again))


def test_no_tokens():
    s = inputs(0, 64, True, "channel")
    got = forward(s, 1.0)
    assert got["out"].shape == got["normed"].shape == (0, 64)
    grads = backward(s, got["out"], 1.0)
    assert grads.dy.shape == (0, 64) and not grads.dpost_weight.any() and not grads.dpre_weight.any() and not grads.dgate.any()


@pytest.mark.parametrize("T,d", [(5, 264), (9, 5000)])
def test_rows_do_not_mix(T, d):
    """A row of zeros is a row of zeros (eps keeps it from 0/0), and an infinity stays in its row."""
    s = inputs(T, d, True, "token")
    s["y"][1].zero_()
    s["residual"][1].zero_()
    clean = forward(s, 1.0)
    assert not clean["out"][1].any() and not clean["normed"][1].any()
    s["y"][T - 1, 3] = float("inf")
    got = forward(s, 1.0)
    for name in got:
        assert torch.equal(got[name][:-1], clean[name][:-1])
    assert not torch.isfinite(got["out"][T - 1].float()).all()
    a, b = backward(s, clean["out"], 1.0), backward(s, got["out"], 1.0)
    assert torch.equal(a.dresidual[:-1], b.dresidual[:-1]) and torch.equal(a.dy[:-1], b.dy[:-1])


@pytest.mark.parametrize("T,d", [(6, 328), (300, 2056)])
def test_nothing_past_the_outputs(T, d):
    s = inputs(T, d, True, "token")

    def inside(shape, dtype=torch.bfloat16):
        n = torch.Size(shape).numel()
        whole = torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda")
        return whole, whole[2048: 2048 + n].view(shape)

    held = {n: inside((T, d)) for n in ("out", "normed", "dresidual", "dy", "dgate")}
    held.update({n: inside((d,), torch.float32) for n in ("dpost_weight", "dpre_weight")})
    v = {n: t[1] for n, t in held.items()}
    got = forward(s, 0.5, out=v["out"], normed=v["normed"])
    backward(s, got["out"], 0.5, grads=moe.BlockNormsGrads(v["dresidual"], v["dy"], v["dpost_weight"], v["dpre_weight"], v["dgate"]))
    want = backward(s, got["out"], 0.5)
    for name, t in want._asdict().items():
        assert torch.equal(v[name], t), name
    for name, (whole, view) in held.items():
        assert (whole[:2048] == 7).all() and (whole[2048 + view.numel():] == 7).all(), name


def test_backward_against_differences():
    T, d = 5, 72
    s = inputs(T, d, True, "channel", seed=3)
    got = forward(s, 0.5)
    grads = backward(s, got["out"], 0.5)
    names = dict(dy="y", dresidual="residual", dpost_weight="post", dpre_weight="pre", dgate="gate")
    at = {n: s[n].double() for n in names.values()}

    def loss(v):
        t = plain_norms.norm(v["y"], EPS)[0] * v["post"]
        out = v["residual"] + 0.5 * v["gate"] * t
        return (out * s["dout"].double()).sum() + (plain_norms.norm(out, EPS)[0] * v["pre"] * s["dnormed"].double()).sum()

    for grad, name in names.items():
        v = torch.randn(at[name].shape, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        h = 1e-6
        slope = (loss({**at, name: at[name] + h * v}) - loss({**at, name: at[name] - h * v})) / (2 * h)
        g = getattr(grads, grad).double()
        # out is rounded before the second norm: a few 2^-8 of each term, of random signs
        assert (slope - (g * v).sum()).abs() <= 4 * plain_norms.H * g.norm() * v.norm(), name


@pytest.mark.parametrize("T,d,gate", [(1, 7168, "channel"), (300, 1000, "token"), (700, 4096, "channel")])
def test_graph_streams_and_repeats(T, d, gate):
    s = inputs(T, d, True, gate)
    ws = torch.full((moe.block_norms_backward_workspace_size(T, d),), 255, dtype=torch.uint8, device="cuda")
    first = forward(s, 0.5)
    grads = backward(s, first["out"], 0.5)
    outs = list(first.values()) + list(grads)

    def call():
        forward(s, 0.5, **first)
        backward(s, first["out"], 0.5, grads=grads, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (5, 6, 7):
        s["y"].copy_(plain.bf16((T, d), 3.0, seed))
        call()
        want = [t.clone() for t in outs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
            got = [t.clone() for t in outs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for t in outs:
            t.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_offsets_past_31_bits():
    """Rows that begin past 2^31 values, against the plain forms of those rows."""
    T, d, n = 300000, 8192, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    y, res, pre, post = rand(T, d), rand(T, d), 1 + 0.1 * rand(d), 1 + 0.1 * rand(d)
    out, normed = moe.block_norms(y, res, pre_weight=pre, post_weight=post, gate=y, scale=0.5)
    for rows in (slice(0, n), slice(T - n, T)):
        check(dict(out=out[rows], normed=normed[rows]),
              plain_norms.forward(y[rows], res[rows], pre, post, y[rows], 0.5, EPS, out[rows]), "forward")
    dout = res
    dout[:-n] = 0  # the sums over the tokens are the last rows'
    got = moe.block_norms_backward(dout, None, y, out, pre_weight=pre, post_weight=post, gate=y, scale=0.5)
    rows = slice(T - n, T)
    want = plain_norms.backward(dout[rows], None, y[rows], out[rows], pre, post, y[rows], 0.5, EPS)
    check(dict(dresidual=got.dresidual[rows], dy=got.dy[rows], dgate=got.dgate[rows], dpost_weight=got.dpost_weight,
               dpre_weight=got.dpre_weight), want, "backward")
