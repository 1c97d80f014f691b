"""The few-token layer (layer_decode): bit for bit what layer_forward gives, with every output
it can write, over layouts, activation formats, widths, adapters and routings that cannot be
certified; beside other work, captured, and on used workspaces; and against the plain fp64
layer."""
import numpy as np
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import synth
from test_gpu_lora import dev_lora, ids_of

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, T, d, L, F, E, k, seed=5, packed=False, act="bf16", bias=None, renormalize=True, adapters=None):
        g = torch.Generator().manual_seed(seed)
        self.T, self.k, self.E = T, k, E
        self.blob = synth.expert_blob(seed, L, F, E, scale_lo=118, scale_hi=121)
        self.cpu = dict(x=plain.bf16((T, d), 1.0, seed), router_w=plain.bf16((E, d), 0.05, seed + 1),
                        latent_down=plain.bf16((L, d), 1.7 * d ** -0.5, seed + 2),
                        latent_up=plain.bf16((d, L), 1.7 * L ** -0.5, seed + 3))
        self.bias = None
        if bias == "expert":
            self.bias = torch.randn(E, generator=g)
        elif bias == "token":
            self.bias = torch.randn((T, E), generator=g)
        self.kw = dict(d_ffn=F, packed=packed, renormalize=renormalize,
                       act_format=moe.ACT_FMT_MXFP8 if act == "mxfp8" else moe.ACT_FMT_BF16)
        self.down = self.up = None
        if adapters:
            N, R, use = adapters
            self.ids = ids_of(T, N, "mixed", seed)
            self.ids[0] = 0
            self.rank = ((torch.arange(N, dtype=torch.int32) * 5) + 3) % (R + 1)
            if use != "up":
                self.down = plain.adapters(N, R, d, L, seed + 4)
            if use != "down":
                self.up = plain.adapters(N, R, L, d, seed + 5)
        self.upload()

    def upload(self):
        self.dev = {n: t.cuda() for n, t in self.cpu.items()}
        self.dev["blob"] = torch.from_numpy(self.blob).cuda()
        if self.kw["packed"]:
            L = self.cpu["latent_down"].shape[0]
            self.dev["blob"] = moe.pack_experts(self.dev["blob"], self.E, L, self.kw["d_ffn"])
        self.kw["bias"] = None if self.bias is None else self.bias.cuda()
        for name, lo in (("lora_down", self.down), ("lora_up", self.up)):
            self.kw[name] = None if lo is None else dev_lora(lo, self.ids, self.rank)

    def routing(self):
        i = lambda *s: torch.full(s, -7, dtype=torch.int32, device="cuda")
        f = lambda *s: torch.full(s, -7.0, dtype=torch.float32, device="cuda")
        return dict(topk_idx=i(self.T, self.k), topk_w=f(self.T, self.k), logits=f(self.T, self.E),
                    expert_counts=i(self.E), expert_offsets=i(self.E + 1), perm=i(self.T * self.k))

    def call(self, fn, routing=None, **kw):
        d = self.dev
        return fn(d["x"], d["router_w"], d["latent_down"], d["latent_up"], d["blob"], self.k, routing=routing,
                  **{**self.kw, **kw})


def bits(t):
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32) if t.dtype == torch.float32 else t


def same_as_forward(layer):
    want_r, got_r = layer.routing(), layer.routing()
    want = layer.call(moe.layer_forward, want_r)
    ws = torch.full((moe.layer_decode_workspace_size(
        moe.make_config(layer.T, *(layer.cpu["latent_down"].shape[::-1]), layer.kw["d_ffn"], layer.E), layer.k,
        *(None if lo is None else moe.LoraArg(None, None, None, None, None, *lo["a"].shape[:2])
          for lo in (layer.down, layer.up))),), 255, dtype=torch.uint8, device="cuda")
    got = layer.call(moe.layer_decode, got_r, workspace=ws)
    for n in want_r:
        assert torch.equal(bits(want_r[n]), bits(got_r[n])), n
    assert torch.equal(bits(want), bits(got))
    return got, got_r


# T, d, L, F, E, k
SIZES = [
    (1, 256, 128, 128, 8, 2),
    (4, 256, 128, 128, 8, 2),
    (1, 32, 128, 128, 1, 1),
    (8, 96, 256, 384, 8, 8),
    (7, 512, 384, 640, 33, 5),
    (1, 1024, 512, 256, 1024, 64),
    (3, 2048, 1024, 512, 64, 16),
    (8, 4096, 3584, 256, 20, 7),
    (2, 8192, 3712, 1280, 6, 3),
    (1, 640, 7168, 4480, 5, 4),
    (5, 160, 256, 7168, 4, 2),
    (8, 224, 7168, 128, 3, 1),
]


@pytest.mark.parametrize("T,d,L,F,E,k", SIZES)
@pytest.mark.parametrize("packed,act", [(False, "bf16"), (True, "bf16"), (True, "mxfp8"), (False, "mxfp8")])
def test_bit_for_bit_layer_forward(T, d, L, F, E, k, packed, act):
    same_as_forward(Layer(T, d, L, F, E, k, packed=packed, act=act))


@pytest.mark.parametrize("T", [1, 2, 8])
@pytest.mark.parametrize("bias", [None, "expert", "token"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_biases_and_weights(T, bias, renormalize):
    same_as_forward(Layer(T, 512, 256, 256, 40, 6, bias=bias, renormalize=renormalize, packed=True))


@pytest.mark.parametrize("T,d,L,F,E,k", SIZES[1:8])
@pytest.mark.parametrize("adapters", [(5, 16, "both"), (3, 128, "up"), (2, 40, "down"), (300, 72, "both")])
def test_adapters(T, d, L, F, E, k, adapters):
    same_as_forward(Layer(T, d, L, F, E, k, packed=True, adapters=adapters))


@pytest.mark.parametrize("T", [1, 3, 8])
def test_ties_and_pruned_experts(T):
    """Selections the certificate cannot decide: equal router rows, all of them, experts at
    -inf with fewer than k left, and tokens holding infinities or NaN."""
    layer = Layer(T, 256, 128, 128, 24, 5)
    layer.cpu["router_w"][3:20] = layer.cpu["router_w"][3]
    layer.upload()
    same_as_forward(layer)
    layer.cpu["router_w"][:] = layer.cpu["router_w"][0]
    layer.upload()
    _, r = same_as_forward(layer)
    assert (r["topk_idx"].cpu() == torch.arange(5)).all()
    layer = Layer(T, 256, 128, 128, 24, 5)
    layer.bias = torch.full((24,), float("-inf"))
    layer.bias[[7, 11]] = 0.5
    layer.upload()
    same_as_forward(layer)
    layer.bias = None
    layer.cpu["x"][0, 3] = float("inf")
    layer.cpu["x"][T - 1, 9] = float("nan")
    layer.upload()
    same_as_forward(layer)
    layer.cpu["x"][:] = 0
    layer.upload()
    same_as_forward(layer)


@pytest.mark.parametrize("T,d,L,F,E,k", [(8, 256, 128, 128, 8, 2), (7, 640, 128, 128, 4, 1), (8, 224, 7168, 7168, 2, 1)])
def test_adapters_of_more_ranks_than_the_layer_is_wide(T, d, L, F, E, k):
    """u of 128 ranks takes more room than the rows it follows in the LDS."""
    layer = Layer(T, d, L, F, E, k, adapters=(5, 128, "up"))
    layer.rank = torch.full((5,), 128, dtype=torch.int32)
    layer.upload()
    same_as_forward(layer)


@pytest.mark.parametrize("word", [-1, 0x7FFFFFFF, 0x7F800001, 0x7F800000, 1, -2 ** 31])
def test_adapter_scales_of_any_bits(word):
    """Scales that are NaN with every payload, infinite, subnormal, a negative zero."""
    layer = Layer(3, 512, 256, 128, 8, 2, adapters=(2, 16, "both"))
    layer.up["scale"] = torch.tensor([word, word], dtype=torch.int32).view(torch.float32)
    layer.upload()
    assert torch.equal(layer.up["scale"].view(torch.int32), torch.tensor([word, word], dtype=torch.int32))
    same_as_forward(layer)


def test_subnormal_and_extreme_scales():
    layer = Layer(4, 256, 128, 256, 8, 2)
    n = 128 * 256 // 2 + 128 * 256 // 32
    s = layer.blob.reshape(8, 3, n)[:, :, 128 * 256 // 2:]
    s[0], s[1, :, ::7], s[2], s[3, :, ::9] = 0, 255, 254, 0
    layer.upload()
    same_as_forward(layer)


@pytest.mark.parametrize("T,act,adapters", [(1, "bf16", None), (5, "mxfp8", None), (8, "bf16", (4, 24, "both"))])
def test_against_the_plain_layer(T, act, adapters):
    """Routing equal; out within its bf16 rounding (2^-8 relative at most, 2^-9 on average) and
    the few one-step differences of h, a and z."""
    layer = Layer(T, 512, 256, 384, 20, 4, act=act, bias="expert", adapters=adapters)
    lo = lambda stack: None if stack is None else (stack, layer.ids, layer.rank)
    c = layer.cpu
    want, idx, w = plain.layer(c["x"], c["router_w"], c["latent_down"], c["latent_up"], layer.blob, 4, 384,
                               bias=layer.bias, act=act, down=lo(layer.down), up=lo(layer.up))
    r = layer.routing()
    got = layer.call(moe.layer_decode, r)
    assert torch.equal(r["topk_idx"].cpu(), idx)
    assert (r["topk_w"].cpu().double() - w).abs().max() <= 2.0 ** -20
    rel = ((got.cpu().double() - want).norm() / want.norm()).item()
    assert rel <= (2.0 ** -8 if act == "bf16" else 2.0 ** -7), rel


def test_two_calls_at_once():
    """Two layers of many blocks on two streams, each call waiting inside itself for its own
    blocks: both end, each as alone."""
    a, b = (Layer(T, 2048, 1024, 1024, 64, 8, seed=s, packed=True) for T, s in ((4, 5), (8, 90)))
    want = [x.call(moe.layer_decode) for x in (a, b)]
    sizes = [moe.layer_decode_workspace_size(moe.make_config(x.T, 2048, 1024, 1024, 64), 8) for x in (a, b)]
    ws = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for x, s, w, o in zip((a, b), streams, ws, outs):
            with torch.cuda.stream(s):
                x.call(moe.layer_decode, workspace=w, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(o), bits(w)) for o, w in zip(outs, want))


@pytest.mark.parametrize("adapters", [None, (3, 16, "both")])
def test_graph_replays(adapters):
    """Captured once, replayed on new tokens and biases with eager work between the replays."""
    layer = Layer(3, 1024, 512, 512, 32, 4, packed=True, bias="expert", adapters=adapters)
    xs = [plain.bf16((3, 1024), 1.0, 200 + i).cuda() for i in range(3)]
    want = []
    for x in xs:
        layer.dev["x"] = x
        r = layer.routing()
        want.append((layer.call(moe.layer_forward, r), r))
    layer.dev["x"] = xs[0].clone()
    r, out = layer.routing(), torch.empty_like(want[0][0])
    ups = [moe._lora(layer.kw[n], 3, *s, xs[0].device) if adapters else None
           for n, s in (("lora_down", (1024, 512)), ("lora_up", (512, 1024)))]
    ws = torch.empty(moe.layer_decode_workspace_size(moe.make_config(3, 1024, 512, 512, 32), 4, *ups),
                     dtype=torch.uint8, device="cuda")
    layer.call(moe.layer_decode, r, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.call(moe.layer_decode, r, out=out, workspace=ws)
    for i in (1, 2, 0, 0, 2):
        layer.dev["x"].copy_(xs[i])
        out.fill_(3)
        r["topk_idx"].fill_(-1)
        graph.replay()
        assert torch.equal(bits(out), bits(want[i][0])), i
        assert torch.equal(r["topk_idx"], want[i][1]["topk_idx"])
        layer.call(moe.layer_decode, workspace=ws)  # the graph's workspace, used between its replays
        torch.cuda.synchronize()


def test_rows_and_bytes_behind_stay():
    layer = Layer(3, 256, 128, 128, 8, 2)
    need = moe.layer_decode_workspace_size(moe.make_config(3, 256, 128, 128, 8), 2)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((5, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    want = layer.call(moe.layer_forward)
    layer.call(moe.layer_decode, out=out[:3], workspace=ws[:need])
    assert torch.equal(out[:3], want) and (out[3:] == 9.0).all() and (ws[need:] == 77).all()


def test_prompt_then_decode_steps_with_adapters():
    """As served: a prompt through layer_forward with its request's adapters, then decode steps
    of several requests through layer_decode, each row as the prompt path gives it."""
    d, L, F, E, k = 512, 256, 256, 32, 4
    layer = Layer(70, d, L, F, E, k, packed=True, adapters=(6, 32, "both"))
    layer.ids = torch.arange(70, dtype=torch.int32) % 7 - 1
    layer.upload()
    prompt = layer.call(moe.layer_forward)
    dv = layer.dev
    for t0 in range(0, 64, 8):
        lo = {n: layer.kw[n]._replace(adapter=layer.kw[n].adapter[t0:t0 + 8].contiguous())
              for n in ("lora_down", "lora_up")}
        step = moe.layer_decode(dv["x"][t0:t0 + 8], dv["router_w"], dv["latent_down"], dv["latent_up"], dv["blob"], k,
                                **{**layer.kw, **lo})
        one = prompt[t0:t0 + 8].double()
        rel = ((step.double() - one).norm() / one.norm()).item()
        assert rel <= 2.0 ** -8, (t0, rel)  # both within their bf16 roundings of the same value
