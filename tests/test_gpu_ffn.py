"""The dense gated block and its backward pass against fp64 forms and differences: every tile that
the sizes choose, odd widths and ragged ends, streams, captured graphs, workspaces, values that
are not finite."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import plain_ffn

pytestmark = pytest.mark.gpu


def weights(d, F, seed=1):
    return (plain.bf16((F, d), d ** -0.5, seed).cuda(), plain.bf16((F, d), d ** -0.5, seed + 1).cuda(),
            plain.bf16((d, F), F ** -0.5, seed + 2).cuda())


def check(got, want, what):
    for name, t in got.items():
        v, bound = want[name]
        off = (t.double() - v).abs() - bound
        assert torch.isfinite(t).all(), (what, name)
        assert off.max() <= 0, (what, name, off.max().item(), (t.double() - v).abs().max().item())


# tokens, width, inner width: single tokens and the few-token tiles, a K shorter than one tile,
# widths that end inside a tile, splits of K, the large tiles
FORWARD = [(1, 8, 8), (1, 256, 344), (1, 7168, 2048), (2, 4096, 512), (3, 72, 1000), (5, 256, 344), (8, 1024, 4096), (9, 512, 512),
           (15, 264, 120), (16, 64, 64), (17, 2048, 1032), (31, 1000, 88), (33, 3584, 7168), (64, 512, 2048), (65, 320, 640),
           (127, 136, 4104), (128, 1024, 1024), (200, 2056, 96), (513, 512, 1528), (1021, 1032, 2056),
           (20, 7168, 512), (64, 1032, 72), (130, 4096, 264), (200, 2048, 1928),
           (2048, 520, 8200), (4096, 4096, 1024), (3600, 7168, 3600)]  # the last: tiles of 224 columns, cut


@pytest.mark.parametrize("T,d,F", FORWARD)
def test_forward(T, d, F):
    x, (wg, wu, wd) = plain.bf16((T, d), 1.0, T).cuda(), weights(d, F)
    want = plain_ffn.forward(x, wg, wu, wd)
    out = moe.gated_ffn(x, wg, wu, wd)
    check(dict(out=out), want, (T, d, F))
    kept = [torch.full((T, F), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    again = moe.gated_ffn(x, wg, wu, wd, gate=kept[0], up=kept[1])
    assert torch.equal(out, again)  # keeping changes nothing
    check(dict(gate=kept[0], up=kept[1]), want, (T, d, F))


BACKWARD = [(1, 8, 8), (1, 512, 264), (5, 64, 128), (33, 136, 72), (77, 512, 1000), (128, 128, 128), (129, 1032, 520),
            (11, 3952, 72), (65, 2056, 264), (100, 1928, 1000), (300, 256, 2056), (1021, 640, 1528), (3001, 72, 136), (5000, 344, 520),
             (2048, 2048, 2048), (4100, 264, 4104), (1000, 4096, 4096), (3900, 3592, 7176)]


@pytest.mark.parametrize("T,d,F", BACKWARD)
def test_backward(T, d, F):
    x, dout = plain.bf16((T, d), 1.0, T).cuda(), plain.bf16((T, d), 0.01, T + 1).cuda()
    wg, wu, wd = weights(d, F)
    gate, up = plain.bf16((T, F), 1.5, 7).cuda(), plain.bf16((T, F), 1.0, 8).cuda()
    got = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
    check(got._asdict(), plain_ffn.backward(dout, x, wg, wu, wd, gate, up), (T, d, F))
    half = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dw=False)
    assert half.dw_gate is None and torch.equal(half.dx, got.dx)
    half = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dx=False)
    assert half.dx is None and torch.equal(half.dw_gate, got.dw_gate) and torch.equal(half.dw_down, got.dw_down)


@pytest.mark.parametrize("T,d,F", [(1, 64, 64), (1, 4096, 8192), (2, 1032, 24576), (3, 512, 1000), (4, 2048, 10240)])
def test_up_to_four_tokens_keep_the_inner_values(T, d, F):
    """a stays fp32 there: no rounding of it.  (2, .., 24576) does not fit and rounds."""
    x, (wg, wu, wd) = plain.bf16((T, d), 1.0, T).cuda(), weights(d, F)
    want = plain_ffn.forward(x, wg, wu, wd, inner=2.0 ** -8 if F == 24576 else 0.0)
    check(dict(out=moe.gated_ffn(x, wg, wu, wd)), want, (T, d, F))


@pytest.mark.parametrize("T,d,F", [(1, 64, 64), (1, 1000, 520), (7, 4104, 136), (33, 136, 2056), (63, 512, 1000), (64, 1024, 512)])
def test_backward_of_few_tokens_keeps_two_halves(T, d, F):
    """a, dG and dU in two halves: the low one, at most 2^-8 of the value, is off by 2^-8 of itself."""
    x, dout = plain.bf16((T, d), 1.0, T).cuda(), plain.bf16((T, d), 0.01, T + 1).cuda()
    wg, wu, wd = weights(d, F)
    gate, up = plain.bf16((T, F), 1.5, 7).cuda(), plain.bf16((T, F), 1.0, 8).cuda()
    got = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
    check(got._asdict(), plain_ffn.backward(dout, x, wg, wu, wd, gate, up, inner=2.0 ** -16), (T, d, F))


def test_halves_of_values_that_overflow():
    """An inner gradient past bf16's range is infinite, as one rounded once is, and not NaN."""
    T, d, F = 3, 64, 64
    x, (wg, wu, wd) = plain.bf16((T, d), 1.0, 1).cuda().abs() + 1, weights(d, F)
    big = torch.full((T, d), 2.0 ** 120, dtype=torch.bfloat16, device="cuda")
    gate = torch.full((T, F), 2.0 ** 6, dtype=torch.bfloat16, device="cuda")  # silu(g) = g, its derivative 1
    up = torch.full((T, F), 2.0 ** 6, dtype=torch.bfloat16, device="cuda")
    wd = wd.abs() + 1  # dA above 2^126, dU and dG above 2^132
    got = moe.gated_ffn_backward(big, x, wg.abs() + 1, wu.abs() + 1, wd, gate, up)
    for t in got:  # dw_down: 3 2^120 2^12
        assert (t == float("inf")).all()


def test_backward_against_differences():
    """The gradient of L = sum(out * dout) along a direction, against L's difference in fp64."""
    T, d, F = 9, 64, 96
    x, dout = plain.bf16((T, d), 1.0, 3).cuda(), plain.bf16((T, d), 1.0, 4).cuda()
    w = weights(d, F)
    gate, up = torch.empty((2, T, F), dtype=torch.bfloat16, device="cuda")
    moe.gated_ffn(x, *w, gate=gate, up=up)
    got = moe.gated_ffn_backward(dout, x, *w, gate, up)

    def loss(x, wg, wu, wd):
        g = x @ wg.T
        return ((g * plain_ffn.sigmoid(g) * (x @ wu.T)) @ wd.T * dout.double()).sum()

    at = [t.double() for t in (x, *w)]
    for i, grad in enumerate(got):
        v = torch.randn(at[i].shape, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
        h = 1e-6
        up_, down_ = list(at), list(at)
        up_[i], down_[i] = at[i] + h * v, at[i] - h * v
        slope = (loss(*up_) - loss(*down_)) / (2 * h)
        # kept g and u are bf16 too: each gradient is a sum of terms off by a few 2^-8 with random signs
        assert (slope - (grad.double() * v).sum()).abs() <= 4 * plain_ffn.H * (grad.double().norm() * v.norm())


def test_no_tokens():
    wg, wu, wd = weights(64, 72)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 72), dtype=torch.bfloat16, device="cuda")
    assert moe.gated_ffn(x, wg, wu, wd).shape == (0, 64)
    got = moe.gated_ffn_backward(x, x, wg, wu, wd, k, k)
    assert got.dx.shape == (0, 64) and not got.dw_gate.any() and not got.dw_up.any() and not got.dw_down.any()


@pytest.mark.parametrize("T,d,F", [(1, 512, 256), (6, 256, 344), (40, 512, 2048), (300, 264, 520), (2048, 2048, 2048)])
def test_nothing_past_the_outputs(T, d, F):
    """Rows and columns past the ends stay as they were, and what stands past the inputs is not read."""
    def inside(shape, fill):
        n = shape[0] * shape[1]
        whole = torch.full((n + 16384,), fill, dtype=torch.bfloat16, device="cuda")
        return whole, whole[8192: 8192 + n].view(shape)

    x, w = plain.bf16((T, d), 1.0, 1).cuda(), weights(d, F)
    dout = plain.bf16((T, d), 0.01, 2).cuda()
    nan = float("nan")
    held = []
    for t in (x, dout, *w):
        whole, view = inside(t.shape, nan)
        view.copy_(t)
        held.append(view)
    xs, ds, *ws = held
    outs = {n: inside(s, 7.0) for n, s in dict(out=(T, d), gate=(T, F), up=(T, F), dx=(T, d), dw_gate=(F, d),
                                                dw_up=(F, d), dw_down=(d, F)).items()}
    v = {n: t[1] for n, t in outs.items()}
    moe.gated_ffn(xs, *ws, out=v["out"], gate=v["gate"], up=v["up"])
    moe.gated_ffn_backward(ds, xs, *ws, v["gate"], v["up"],
                           out=moe.GatedFfnGrads(v["dx"], v["dw_gate"], v["dw_up"], v["dw_down"]))
    want = plain_ffn.forward(x, *w)
    check({n: v[n] for n in ("out", "gate", "up")}, want, "forward")
    check({n: v[n] for n in ("dx", "dw_gate", "dw_up", "dw_down")},
          plain_ffn.backward(dout, x, *w, v["gate"], v["up"]), "backward")
    for n, (whole, view) in outs.items():
        assert (whole[:8192] == 7).all() and (whole[8192 + view.numel():] == 7).all(), n


@pytest.mark.parametrize("T", [1, 3, 20, 50, 200, 600])
def test_rows_do_not_mix(T):
    """An infinity in one token's row reaches that token's results only."""
    x, w = plain.bf16((T, 264), 1.0, 1).cuda(), weights(264, 328)
    clean = moe.gated_ffn(x, *w)
    x[T // 2, 5] = float("inf")
    got = moe.gated_ffn(x, *w)
    others = [t for t in range(T) if t != T // 2]
    assert torch.equal(got[others], clean[others]) and not torch.isfinite(got[T // 2]).any()


def test_large_values():
    """Gates far from zero: silu falls to 0 and rises to g, and its slope to 0 and 1."""
    T, d, F = 16, 64, 64
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.linspace(-300, 300, T).cuda()
    x[:, 1] = 1.0
    wg, wu, wd = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((F, d), (F, d), (d, F)))
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    wd.fill_(1.0)
    gate, up = torch.empty((2, T, F), dtype=torch.bfloat16, device="cuda")
    out = moe.gated_ffn(x, wg, wu, wd, gate=gate, up=up)
    check(dict(out=out), plain_ffn.forward(x, wg, wu, wd), "large")
    dout = torch.ones_like(x)
    check(moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)._asdict(),
          plain_ffn.backward(dout, x, wg, wu, wd, gate, up), "large")


@pytest.mark.parametrize("T,d,F", [(1, 512, 264), (40, 512, 2048), (700, 512, 520)])
def test_graph_streams_and_repeats(T, d, F):
    """A training step captured into a graph and replayed on new contents, and one on a side stream,
    give the eager call's bits; the workspace needs no clearing and serves both passes."""
    x, dout, w = plain.bf16((T, d), 1.0, 1).cuda(), plain.bf16((T, d), 0.01, 2).cuda(), weights(d, F)
    ws = torch.full((max(moe.gated_ffn_workspace_size(T, d, F), moe.gated_ffn_workspace_size(T, d, F, True)),), 255,
                    dtype=torch.uint8, device="cuda")
    gate, up = torch.empty((2, T, F), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    grads = moe.GatedFfnGrads(torch.empty_like(x), *(torch.empty_like(t) for t in w))

    def step(stream=None):
        moe.gated_ffn(x, *w, out=out, gate=gate, up=up, workspace=ws, stream=stream)
        moe.gated_ffn_backward(dout, x, *w, gate, up, out=grads, workspace=ws, stream=stream)
        return [t.clone() for t in (out, gate, up, *grads)]

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.gated_ffn(x, *w, out=out, gate=gate, up=up, workspace=ws)
        moe.gated_ffn_backward(dout, x, *w, gate, up, out=grads, workspace=ws)
    for seed in (5, 6, 7):
        x.copy_(plain.bf16((T, d), 1.0, seed))
        want = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for t in (out, gate, up, *grads):
            t.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, gate, up, *grads), want))


def test_offsets_past_31_bits():
    """Rows that begin past 2^31 values of the inner tensors, against the same rows alone."""
    T, d, F, n = 140000, 64, 16384, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape, std=1.0: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)
    x, dout, (wg, wu, wd) = rand(T, d), rand(T, d, std=0.01), weights(d, F)
    gate, up = rand(T, F), rand(T, F)
    out = moe.gated_ffn(x, wg, wu, wd, gate=gate, up=up)
    want = plain_ffn.forward(x[-n:], wg, wu, wd)
    check(dict(out=out[-n:], gate=gate[-n:], up=up[-n:]), want, "last rows")
    check(dict(out=out[:n]), plain_ffn.forward(x[:n], wg, wu, wd), "first rows")
    dx = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dw=False).dx
    for rows in (slice(0, n), slice(T - n, T)):
        back = plain_ffn.backward(dout[rows], x[rows], wg, wu, wd, gate[rows], up[rows])
        check(dict(dx=dx[rows]), back, "backward")
    # only the last rows have a gradient: the sums over all tokens are theirs
    dout[:-n] = 0
    got = moe.gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dx=False)
    rows = slice(T - n, T)
    back = plain_ffn.backward(dout[rows], x[rows], wg, wu, wd, gate[rows], up[rows])
    # a sum over T tokens, of which all but n are zeros, rounds no more often than one over n
    check(dict(dw_gate=got.dw_gate, dw_up=got.dw_up, dw_down=got.dw_down), back, "weights")


def test_two_calls_at_once():
    """Calls of different sizes on two streams, each with a workspace of its own: the bits of each alone."""
    sizes = [(1100, 1032, 2056), (77, 512, 1000)]
    made = []
    for T, d, F in sizes:
        x, dout, w = plain.bf16((T, d), 1.0, 1).cuda(), plain.bf16((T, d), 0.01, 2).cuda(), weights(d, F)
        gate, up = torch.empty((2, T, F), dtype=torch.bfloat16, device="cuda")
        made.append((x, dout, w, gate, up))

    def call(x, dout, w, gate, up, stream=None):
        out = moe.gated_ffn(x, *w, gate=gate, up=up, stream=stream)
        return [out, *moe.gated_ffn_backward(dout, x, *w, gate, up, stream=stream)]

    want = [call(*m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        got = [call(*m, stream=s) for _ in range(3) for m, s in zip(made, streams)]
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
