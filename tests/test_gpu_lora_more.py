"""Adapters where the other tests do not go: the layer at 9 to 31 tokens, stacks of hundreds of which a
call meets a few, tokens without an adapter on large matrices."""
import pytest
import torch

import mxfp4_expert_gemm_amd as moe
import plain
from test_gpu_lora import check, dev_lora, ids_of, layer_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [9, 16, 31])
@pytest.mark.parametrize("use", ["both", "up", "down"])
@pytest.mark.parametrize("packed,act", [(False, "bf16"), (True, "mxfp8")])
def test_layer_at_9_to_31_tokens(T, use, packed, act):
    """Routing equal, out within bf16's rounding (2^-8 relative at most, 2^-9 on average) and the few
    one-step differences of h, a and z."""
    d, L, F, E, k, N, R = 512, 256, 128, 10, 3, 5, 40
    blob, w, down, up = layer_inputs(T, d, L, F, E, N, R, 60)
    ids = ids_of(T, N, "mixed", T)
    rank = torch.tensor([40, 0, 9, 33, 16], dtype=torch.int32)
    on = dict(down=use != "up", up=use != "down")
    want, idx, wt = plain.layer(w["x"], w["router_w"], w["latent_down"], w["latent_up"], blob, k, F, act=act,
                                down=(down, ids, rank) if on["down"] else None, up=(up, ids, rank) if on["up"] else None)
    db = torch.from_numpy(blob).cuda()
    if packed:
        db = moe.pack_experts(db, E, L, F)
    r = dict(topk_idx=torch.empty((T, k), dtype=torch.int32, device="cuda"))
    got = moe.layer_forward(*(w[n].cuda() for n in ("x", "router_w", "latent_down", "latent_up")), db, k, d_ffn=F,
                            packed=packed, act_format=moe.ACT_FMT_MXFP8 if act == "mxfp8" else moe.ACT_FMT_BF16, routing=r,
                            lora_down=dev_lora(down, ids, rank) if on["down"] else None,
                            lora_up=dev_lora(up, ids, rank) if on["up"] else None)
    assert torch.equal(r["topk_idx"].cpu(), idx)
    rel = ((got.cpu().double() - want).norm() / want.norm()).item()
    assert rel <= (2.0 ** -8 if act == "bf16" else 2.0 ** -7), rel


@pytest.mark.parametrize("N", [300, 512, 1024])
@pytest.mark.parametrize("T,n_in,n_out", [(600, 1024, 200), (1021, 2048, 130), (4096, 512, 96)])
def test_large_stacks_of_which_few_are_met(T, n_in, n_out, N):
    R = 16
    x, W = plain.bf16((T, n_in), 1.0, 1), plain.bf16((n_out, n_in), 0.03, 2)
    lo = plain.adapters(N, R, n_in, n_out, 3)
    met = torch.tensor([0, 7, N // 2, N - 2, N - 1], dtype=torch.int32)
    for ids in (met[torch.arange(T) % 5], met[torch.arange(T) * 5 // T], torch.full((T,), N - 1, dtype=torch.int32)):
        check(moe.linear_lora(x.cuda(), W.cuda(), dev_lora(lo, ids)), x, W, lo, ids, None, (T, N))


@pytest.mark.parametrize("T", [1, 4, 5, 17, 31, 32, 33])
@pytest.mark.parametrize("n_in,n_out", [(7168, 3584), (3584, 7168)])
def test_rows_without_an_adapter_on_large_matrices(T, n_in, n_out):
    """Such a row is the projection alone, by the kernels the call takes: bit for bit linear_bf16's row
    in a call of as many tokens, or, from 5 to 31 tokens, in one of 32."""
    x, W = plain.bf16((T, n_in), 1.0, 1).cuda(), plain.bf16((n_out, n_in), 0.02, 2).cuda()
    lo = plain.adapters(2, 16, n_in, n_out, 3)
    ids = torch.full((T,), -1, dtype=torch.int32)
    if T > 2:
        ids[1] = 1
    got = moe.linear_lora(x, W, dev_lora(lo, ids))
    as_many = torch.zeros((32, n_in), dtype=torch.bfloat16, device="cuda")
    as_many[:min(T, 32)] = x[:32]
    want = moe.linear_bf16(as_many, W)[:T] if 5 <= T < 32 else moe.linear_bf16(x, W)
    none = [t for t in range(T) if ids[t] < 0]
    assert torch.equal(got[none], want[none])


def test_no_tokens():
    """Calls without a token return empty outputs and touch nothing."""
    d, L, F, E, k, N, R = 256, 128, 128, 8, 2, 3, 8
    blob, w, down, up = layer_inputs(0, d, L, F, E, N, R, 5)
    ids = torch.zeros(0, dtype=torch.int32)
    dev = {n: t.cuda() for n, t in w.items()}
    lo = dict(lora_down=dev_lora(down, ids), lora_up=dev_lora(up, ids))
    assert moe.linear_lora(dev["x"], dev["latent_down"], lo["lora_down"]).shape == (0, L)
    for fn in (moe.layer_forward, moe.layer_decode):
        out = fn(dev["x"], dev["router_w"], dev["latent_down"], dev["latent_up"], torch.from_numpy(blob).cuda(), k, d_ffn=F, **lo)
        assert out.shape == (0, d)
    torch.cuda.synchronize()
