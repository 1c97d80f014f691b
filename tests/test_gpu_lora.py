"""Adapters of many requests beside a shared projection (linear_lora, and the layer with
adapters) against plain fp64 forms: every kernel the sizes choose, ids and ranks at their
ends, rows that must not touch each other, streams, captured graphs and repeated calls."""
import numpy as np
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
import synth

pytestmark = pytest.mark.gpu


def ids_of(T, N, order, seed):
    g = torch.Generator().manual_seed(seed + 3)
    ids = torch.randint(-1, N + 1, (T,), generator=g, dtype=torch.int32)  # -1 and N: no adapter
    return ids.sort()[0] if order == "segments" else ids


def dev_lora(lo, ids, rank=None):
    return moe.Lora(lo["a"].cuda(), lo["b"].cuda(), lo["scale"].float().cuda(), ids.cuda(),
                    None if rank is None else rank.cuda())


def check(got, x, W, lo, ids, rank, what):
    v, S = plain.linear(x.cuda(), W.cuda(), {n: t.cuda() for n, t in lo.items()}, ids.cuda(), rank)
    off = (got.double() - v).abs() - plain.linear_bound(v, S, x.shape[1])
    assert off.max() <= 0, (what, off.max().item())


# T, n_in, n_out, adapters, max rank, order, ragged ranks.  Below 32 tokens (for large matrices
# below 5; or n_in no multiple of 64) the GEMV with 4, 2 or 1 tokens a block; then the small tiles,
# the 128 x 128 ones from 384 of them on, and the LDS-direct ones from 768; the first product
# by rows up to 512 tokens and 16384 (token, rank) pairs, grouped above.
CASES = [
    (1, 32, 1, 1, 8, "mixed", False),
    (1, 7168, 3584, 3, 16, "mixed", True),
    (2, 3584, 7168, 5, 128, "mixed", True),
    (3, 8192, 65, 2, 24, "mixed", False),
    (5, 512, 130, 7, 40, "mixed", True),
    (4, 7168, 3584, 3, 16, "mixed", False),
    (5, 7168, 3584, 3, 40, "mixed", True),
    (9, 8192, 1025, 9, 8, "mixed", False),
    (17, 3584, 7168, 17, 128, "mixed", True),
    (31, 7168, 3584, 4, 16, "segments", True),
    (31, 8160, 700, 4, 16, "mixed", True),
    (16, 256, 128, 4, 8, "mixed", True),
    (31, 4096, 64, 1024, 16, "mixed", False),
    (32, 64, 33, 3, 8, "segments", True),
    (33, 3584, 1000, 9, 64, "mixed", True),
    (64, 7168, 3584, 64, 16, "mixed", True),
    (65, 128, 2049, 6, 128, "mixed", True),
    (100, 96, 77, 5, 64, "mixed", True),
    (130, 2048, 512, 3, 32, "segments", True),
    (257, 1024, 300, 17, 48, "mixed", True),
    (300, 96, 129, 300, 128, "mixed", True),
    (1021, 640, 1100, 5, 128, "segments", True),
    (1000, 2560, 96, 40, 56, "mixed", True),
    (200, 192, 130, 20, 128, "segments", True),
    (512, 320, 257, 33, 32, "mixed", True),
    (513, 320, 257, 33, 8, "mixed", False),
    (1500, 320, 5000, 9, 40, "segments", True),
    (2049, 128, 3201, 600, 128, "mixed", True),
    (4096, 128, 3201, 1000, 16, "mixed", True),
    (4099, 576, 3250, 6, 96, "segments", True),
]


@pytest.mark.parametrize("T,n_in,n_out,N,R,order,ragged", CASES)
def test_linear_lora_against_fp64(T, n_in, n_out, N, R, order, ragged):
    x, W = plain.bf16((T, n_in), 1.0, 1), plain.bf16((n_out, n_in), 0.02, 2)
    lo = plain.adapters(N, R, n_in, n_out, 3)
    ids = ids_of(T, N, order, T)
    rank = None
    if ragged:  # every length from none to all, and values past both ends
        rank = (torch.arange(N, dtype=torch.int32) * 5) % (R + 3) - 1
    got = moe.linear_lora(x.cuda(), W.cuda(), dev_lora(lo, ids, rank))
    check(got, x, W, lo, ids, rank, (T, n_in, n_out))


@pytest.mark.parametrize("T", [1, 7, 40, 300, 2000])
def test_no_adapter_is_the_projection_bit_for_bit(T):
    x, W = plain.bf16((T, 512), 1.0, 1).cuda(), plain.bf16((200, 512), 0.05, 2).cuda()
    lo = plain.adapters(4, 16, 512, 200, 3)
    for ids in (torch.full((T,), -1, dtype=torch.int32), torch.full((T,), 2 ** 31 - 1, dtype=torch.int32)):
        assert torch.equal(moe.linear_lora(x, W, dev_lora(lo, ids)), moe.linear_bf16(x, W))
    none = torch.zeros(4, dtype=torch.int32)  # every rank 0
    assert torch.equal(moe.linear_lora(x, W, dev_lora(lo, ids_of(T, 4, "mixed", 1), none)), moe.linear_bf16(x, W))


@pytest.mark.parametrize("T,R", [(6, 16), (48, 24), (300, 40)])
def test_one_request_never_reaches_another(T, R):
    """Adapter 1 holds infinities and NaN and token 2 too: every other row is as without them.
    Ranks past an adapter's own hold NaN: never used."""
    n_in, n_out, N = 256, 96, 4
    x, W = plain.bf16((T, n_in), 1.0, 1), plain.bf16((n_out, n_in), 0.05, 2)
    lo = plain.adapters(N, R, n_in, n_out, 3)
    ids = torch.arange(T, dtype=torch.int32) % N
    rank = torch.tensor([R - 3, R, 1, R - 8], dtype=torch.int32)
    clean = moe.linear_lora(x.cuda(), W.cuda(), dev_lora(lo, ids, rank))
    check(clean, x, W, lo, ids, rank, "clean")
    for i in range(N):
        lo["a"][i, int(rank[i]):] = float("nan")
        lo["b"][i, :, int(rank[i]):] = float("nan")
    assert torch.equal(moe.linear_lora(x.cuda(), W.cuda(), dev_lora(lo, ids, rank)), clean)
    lo["a"][1, 0, 5] = float("inf")
    lo["b"][1, 3] = float("nan")
    x[2, 7] = float("inf")
    got = moe.linear_lora(x.cuda(), W.cuda(), dev_lora(lo, ids, rank))
    others = [t for t in range(T) if t % N != 1 and t != 2]
    assert torch.equal(got[others], clean[others])
    assert not torch.isfinite(got[1].float()).any() and not torch.isfinite(got[2].float()).any()


@pytest.mark.parametrize("T,R", [(3, 16), (64, 16), (600, 32)])
def test_graph_streams_and_repeats(T, R):
    """A captured call replayed with new contents, a side stream and a second call agree with
    the eager one bit for bit; the workspace needs no clearing."""
    n_in, n_out, N = 1024, 640, 5
    lo = plain.adapters(N, R, n_in, n_out, 3)
    W = plain.bf16((n_out, n_in), 0.03, 2).cuda()
    xs = [plain.bf16((T, n_in), 1.0, 10 + i).cuda() for i in range(3)]
    lds = [dev_lora(lo, ids_of(T, N, "mixed", i)) for i in range(3)]
    want = [moe.linear_lora(x, W, l) for x, l in zip(xs, lds)]
    ws = torch.full((moe.linear_lora_workspace_size(T, n_in, N, R),), 255, dtype=torch.uint8, device="cuda")
    x, l, out = xs[0].clone(), lds[0]._replace(adapter=lds[0].adapter.clone()), torch.empty_like(want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.linear_lora(x, W, l, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.linear_lora(x, W, l, out=out, workspace=ws)
    for i in (1, 2, 0, 2):
        x.copy_(xs[i])
        l.adapter.copy_(lds[i].adapter)
        out.fill_(7)
        graph.replay()
        assert torch.equal(out, want[i]), i
        assert torch.equal(moe.linear_lora(xs[0], W, lds[0]), want[0])
        torch.cuda.synchronize()


def test_rows_behind_the_batch_stay():
    T, n_in, n_out, N, R = 37, 128, 65, 3, 16
    x, W = plain.bf16((T, n_in), 1.0, 1), plain.bf16((n_out, n_in), 0.05, 2)
    lo = plain.adapters(N, R, n_in, n_out, 3)
    ids = ids_of(T, N, "mixed", 1)
    need = moe.linear_lora_workspace_size(T, n_in, N, R)
    out = torch.full((T + 3, n_out), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    moe.linear_lora(x.cuda(), W.cuda(), dev_lora(lo, ids), out=out[:T], workspace=ws[:need])
    assert (out[T:] == 5.0).all() and (ws[need:] == 77).all()
    check(out[:T], x, W, lo, ids, None, "rows")


def layer_inputs(T, d, L, F, E, N, R, seed):
    blob = synth.expert_blob(seed, L, F, E, scale_lo=118, scale_hi=121)
    w = dict(x=plain.bf16((T, d), 1.0, seed), router_w=plain.bf16((E, d), 0.05, seed + 1),
             latent_down=plain.bf16((L, d), 0.05, seed + 2), latent_up=plain.bf16((d, L), 0.05, seed + 3))
    down, up = plain.adapters(N, R, d, L, seed + 4), plain.adapters(N, R, L, d, seed + 5)
    return blob, w, down, up


@pytest.mark.parametrize("T,use", [(1, "both"), (3, "up"), (8, "down"), (40, "both"), (90, "both")])
@pytest.mark.parametrize("packed,act", [(False, "bf16"), (True, "mxfp8")])
def test_layer_with_adapters_against_fp64(T, use, packed, act):
    """Routing equal (the adapters do not reach the router), out within bf16's rounding: its
    own (2^-8 relative at most, 2^-9 on average) and the few one-step differences of h, a and z."""
    d, L, F, E, k, N, R = 256, 128, 256, 12, 3, 4, 24
    blob, w, down, up = layer_inputs(T, d, L, F, E, N, R, 50)
    ids = ids_of(T, N, "mixed", T)
    rank = torch.tensor([24, 0, 9, 16], dtype=torch.int32)
    want, idx, wt = plain.layer(w["x"], w["router_w"], w["latent_down"], w["latent_up"], blob, k, F, act=act,
                                down=(down, ids, rank) if use != "up" else None,
                                up=(up, ids, rank) if use != "down" else None)
    dev = {n: t.cuda() for n, t in w.items()}
    db = torch.from_numpy(blob).cuda()
    if packed:
        db = moe.pack_experts(db, E, L, F)
    routing = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                   topk_w=torch.empty((T, k), dtype=torch.float32, device="cuda"))
    got = moe.layer_forward(dev["x"], dev["router_w"], dev["latent_down"], dev["latent_up"], db, k, d_ffn=F,
                            packed=packed, act_format=moe.ACT_FMT_MXFP8 if act == "mxfp8" else moe.ACT_FMT_BF16,
                            routing=routing, lora_down=dev_lora(down, ids, rank) if use != "up" else None,
                            lora_up=dev_lora(up, ids, rank) if use != "down" else None)
    assert torch.equal(routing["topk_idx"].cpu(), idx)
    assert (routing["topk_w"].cpu().double() - wt).abs().max() <= 2.0 ** -20
    rel = ((got.cpu().double() - want).norm() / want.norm()).item()
    assert rel <= 2.0 ** -8 if act == "bf16" else rel <= 2.0 ** -7, rel
    plain_out = moe.layer_forward(dev["x"], dev["router_w"], dev["latent_down"], dev["latent_up"], db, k, d_ffn=F,
                                  packed=packed, act_format=moe.ACT_FMT_MXFP8 if act == "mxfp8" else moe.ACT_FMT_BF16)
    on = ((ids >= 0) & (ids < N) & (rank[ids.clamp(0, N - 1).long()] > 0)).numpy()
    same = (got == plain_out).all(1).cpu().numpy()
    assert same[~on].all() and not same[on].any()


def test_layer_with_adapters_and_shared_experts():
    """The shared experts' fp32 rows and the adapters' term meet in one rounding: the layer
    with both less the layer with either alone is what the two add."""
    T, d, L, F, E, k, N, R, FS = 6, 256, 128, 128, 8, 2, 3, 16, 128
    blob, w, down, up = layer_inputs(T, d, L, F, E, N, R, 80)
    shared = synth.expert_blob(9, d, FS, 2, scale_lo=118, scale_hi=121)
    ids = torch.tensor([0, 1, 2, -1, 0, 2], dtype=torch.int32)
    dev = {n: t.cuda() for n, t in w.items()}
    args = (dev["x"], dev["router_w"], dev["latent_down"], dev["latent_up"], torch.from_numpy(blob).cuda(), k)
    sh = dict(shared_blob=torch.from_numpy(shared).cuda(), num_shared=2, d_ffn_shared=FS)
    lo = dict(lora_up=dev_lora(up, ids))
    both = moe.layer_forward(*args, d_ffn=F, **sh, **lo).double()
    no_lora, no_shared, neither = (moe.layer_forward(*args, d_ffn=F, **kw).double() for kw in (sh, lo, {}))
    off = (both - no_lora - no_shared + neither).abs()
    # four roundings of at most 2^-8 of their own values
    assert (off <= 2.0 ** -8 * (both.abs() + no_lora.abs() + no_shared.abs() + neither.abs()) + 1e-6).all()
    assert torch.equal(both[3], no_lora[3])
