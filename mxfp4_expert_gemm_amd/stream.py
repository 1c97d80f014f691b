"""Layers whose experts do not all fit in HBM: prefix pinning and per-call streaming.

A Kimi K3 has 92 routed layers with 896 experts of 17,547,264 bytes each: 15.7 GB of
experts per layer and 1.45 TB in all (in-c post, section on how the memory requirement
shrinks), five times the 288 GB of one MI355X.  Two facts of that post decide the design:

* Only the experts a token routes to are needed: 16 of 896 per layer and token.  A layer
  whose records stay in pinned host memory runs through `layer_forward_streamed`, which
  copies just the routed records into HBM slots on the device before its expert kernels.
* Layers are visited in the same order for every token, a cyclic scan.  For that pattern
  a least-recently-used cache with fewer slots than layers never hits (the post's example:
  93 layers, 90 slots, hit rate 0), while pinning the first N layers guarantees N of every
  pass (90/93 = 96.8%).  So the first N layers keep their experts in HBM for good and the
  others stream (section on streaming the trunk, which applies it to the dense weights).

`plan_prefix` sizes N for an HBM budget, `cache_hits` replays the scan for either policy,
and `LayerStack` runs a stack with the first N layers resident and the rest streamed: each
layer on an input of its own (`step`), or as the blocks of one residual stream with the norms
between them, dense layers among them and a projection of the result (`forward`).
"""
from __future__ import annotations

from collections import OrderedDict
from typing import List, Optional, Sequence, Tuple

import torch

from . import (_BF16, _F32, _I8, NORM_EPS, _at, _shaped, alloc_expert_slots, alloc_workspace, block_norms,
               expert_bytes, gated_ffn, gated_ffn_workspace_size, layer_forward, layer_forward_streamed, linear_bf16,
               linear_int8, make_config, packed_expert_bytes)

_FLT_MAX = torch.finfo(torch.float32).max


def plan_prefix(num_layers: int, layer_expert_bytes: int, hbm_budget_bytes: int, reserved_bytes: int = 0) -> int:
    """Layers whose experts fit in the HBM budget after the reserved bytes (dense weights,
    workspace, slot buffer): the first N are pinned, N = min(num_layers, free // per layer)."""
    if num_layers < 0 or layer_expert_bytes <= 0:
        raise ValueError("num_layers >= 0 and layer_expert_bytes > 0")
    free = hbm_budget_bytes - reserved_bytes
    return max(0, min(num_layers, free // layer_expert_bytes))


def cache_hits(num_layers: int, passes: int, slots: int, policy: str) -> int:
    """Hits over `passes` scans of layers 0..num_layers-1 with `slots` layer-sized slots.
    policy 'lru': least recently used eviction; 'prefix': layers < slots pinned, the rest
    always fetched."""
    if policy == "prefix":
        return passes * min(slots, num_layers)
    if policy != "lru":
        raise ValueError(policy)
    cache: "OrderedDict[int, None]" = OrderedDict()
    hits = 0
    for _ in range(passes):
        for layer in range(num_layers):
            if layer in cache:
                hits += 1
                cache.move_to_end(layer)
                continue
            if slots == 0:
                continue
            if len(cache) >= slots:
                cache.popitem(last=False)
            cache[layer] = None
    return hits


def _dense(layer: dict) -> bool:
    return "w_gate" in layer


class LayerStack:
    """A stack of MoE layers: dense weights in HBM, experts in HBM for the first `pinned`
    layers and in pinned host memory for the others.

    layers: per layer a dict with router_w, latent_down, latent_up (device bf16 tensors)
    and expert_blob_host (pinned host uint8 tensor, E records).  Layers may share tensors
    (the same object is uploaded once).  Every layer call uses one workspace and one slot
    buffer, sized for `num_tokens` tokens.

    A dict with w_gate, w_up and w_down (device bf16 tensors) is a dense layer instead, a gated
    block whose weights stay in HBM; it counts among the pinned layers where it stands among them.
    For `forward`, a layer's dict may hold pre_norm (bf16 [d]: the norm of its input; without it
    the layer takes the stream as it is), post_norm (bf16 [d]: the norm of its result), gate
    (bf16 [d] or [num_tokens, d]) and scale (a number) for its result's way into the stream.
    """

    def __init__(self, layers: Sequence[dict], k: int, d_ffn: int, pinned: int, num_tokens: int, *,
                 packed: bool = False, device="cuda"):
        if not 0 <= pinned <= len(layers):
            raise ValueError("pinned must be in [0, number of layers]")
        self.layers = list(layers)
        self.k, self.d_ffn, self.pinned, self.packed = k, d_ffn, pinned, packed
        self.resident: List[Optional[torch.Tensor]] = []
        uploaded = {}
        self.widths = [lay["w_gate" if _dense(lay) else "router_w"].shape[1] for lay in self.layers]
        for i, lay in enumerate(self.layers):
            if _dense(lay):
                self.resident.append(None)
                continue
            host = lay["expert_blob_host"]
            if host.is_cuda or not host.is_pinned():
                raise ValueError(f"layer {i}: expert_blob_host must be a pinned host tensor")
            if i < pinned:
                key = host.data_ptr()
                if key not in uploaded:
                    uploaded[key] = host.to(device, non_blocking=False)
                self.resident.append(uploaded[key])
            else:
                self.resident.append(None)
        T, self.num_tokens = num_tokens, num_tokens
        self.workspace = self.slots = None
        sparse = [i for i, lay in enumerate(self.layers) if not _dense(lay)]
        if sparse:
            first = self.layers[sparse[0]]
            cfg = make_config(T, self.widths[sparse[0]], first["latent_down"].shape[0], d_ffn, first["router_w"].shape[0], packed=packed)
            self.workspace = alloc_workspace(cfg, k, device)
            self.slots = alloc_expert_slots(cfg, k, device) if pinned <= sparse[-1] else None
        widest = [gated_ffn_workspace_size(T, *reversed(lay["w_gate"].shape)) for lay in self.layers if _dense(lay)]
        self.dense_workspace = torch.empty(max(widest), dtype=torch.uint8, device=device) if widest else None

    def forward_layer(self, i: int, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                      routing: Optional[dict] = None, stream=None) -> torch.Tensor:
        lay = self.layers[i]
        if _dense(lay):
            if routing is not None:
                raise ValueError(f"layer {i} is dense: it routes nothing")
            # of another number of tokens the workspace may be too small
            work = self.dense_workspace if x.shape[0] == self.num_tokens else None
            return gated_ffn(x, lay["w_gate"], lay["w_up"], lay["w_down"], out=out, workspace=work, stream=stream)
        args = (x, lay["router_w"], lay["latent_down"], lay["latent_up"])
        kw = dict(d_ffn=self.d_ffn, bias=lay.get("bias"), out=out, workspace=self.workspace, routing=routing,
                  stream=stream, packed=self.packed)
        if self.resident[i] is not None:
            return layer_forward(*args, self.resident[i], self.k, **kw)
        return layer_forward_streamed(*args, lay["expert_blob_host"], self.k, expert_slots=self.slots, **kw)

    def _check_pass(self, x: torch.Tensor, final_norm: Optional[torch.Tensor], head, eps: float):
        """What forward is given and what the layers hold, before any of it runs: a pass that is refused
        half way has fetched experts for nothing, and the routed layers' calls take their tensors as they are."""
        T, d, device = self.num_tokens, x.shape[-1], x.get_device()

        def fits(name, t, shape, dtypes=_BF16):
            if t.shape != shape or t.dtype not in dtypes or t.get_device() != device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor of shape {shape} on the device of x")

        _shaped("x", x, (T, d))
        if not 0 <= eps <= _FLT_MAX:
            raise ValueError("eps must be a finite fp32 number, 0 or more")
        each = packed_expert_bytes if self.packed else expert_bytes
        sizes = {}
        for i, lay in enumerate(self.layers):
            if self.widths[i] != d:
                raise ValueError(f"layer {i} is {self.widths[i]} wide and the stream {d}")
            for name in ("pre_norm", "post_norm"):
                if lay.get(name) is not None:
                    fits(name, lay[name], (d,))
            gate = lay.get("gate")
            if gate is not None:
                fits("gate", gate, (d,) if gate.dim() == 1 else (T, d))
            if not abs(lay.get("scale", 1.0)) <= _FLT_MAX:
                raise ValueError("scale must be a finite fp32 number")
            if _dense(lay):
                F = lay["w_gate"].shape[0]
                for name, shape in (("w_gate", (F, d)), ("w_up", (F, d)), ("w_down", (d, F))):
                    fits(name, lay[name], shape)
                continue
            E, L = lay["router_w"].shape[0], lay["latent_down"].shape[0]
            fits("router_w", lay["router_w"], (E, d))
            fits("latent_down", lay["latent_down"], (L, d))
            fits("latent_up", lay["latent_up"], (d, L))
            bias = lay.get("bias")
            if bias is not None:
                fits("bias", bias, (E,) if bias.dim() == 1 else (T, E), _F32)
            if L not in sizes:
                sizes[L] = each(L, self.d_ffn)
            blob = lay["expert_blob_host"]
            if blob.numel() * blob.element_size() < E * sizes[L]:
                raise ValueError(f"layer {i}: expert_blob_host is smaller than {E} experts")
        if final_norm is not None:
            fits("final_norm", final_norm, (d,))
        if head is not None:
            if final_norm is None:
                raise ValueError("head needs final_norm")
            if isinstance(head, torch.Tensor):
                fits("head", head, (head.shape[0], d))
            else:
                W, w_scale = head
                fits("head", W, (W.shape[0], d), _I8)
                fits("the head's scales", w_scale, (W.shape[0],), _F32)
                if d % 16:
                    raise ValueError("a head in 8 bits takes widths that are multiples of 16")

    def forward(self, x: torch.Tensor, *, final_norm: Optional[torch.Tensor] = None, head=None, eps: float = NORM_EPS,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """One pass of a residual stream over the stack, x bf16 [num_tokens, d] its start: for each layer
            stream = stream + scale gate norm(layer(norm(stream) pre_norm)) post_norm
        with what its dict holds of them; attention, which comes between them in a model, is not part of
        this path.  One call to block_norms ends a layer and begins the next.  Returns (stream, None),
        with final_norm (bf16 [d]) the normed stream as the second, and with head the projection of it:
        a bf16 [n_out, d] for linear_bf16 or (codes, scales) for linear_int8.  Shapes, types and places are
        checked before anything runs."""
        self._check_pass(x, final_norm, head, eps)
        residual = y = None
        done = {}
        for i, lay in enumerate(self.layers + [{"pre_norm": final_norm}]):
            pre = lay.get("pre_norm")
            if y is None:  # the start: x itself, of which there is at most the norm
                residual, h = x, x
                if pre is not None:
                    h = block_norms(None, x, pre_weight=pre, eps=eps, stream=stream)[1]
            else:  # the first result takes a place of its own, the others are added there
                into = None if residual is x else residual
                residual, h = block_norms(y, residual, pre_weight=pre, post_weight=done.get("post_norm"),
                                          gate=done.get("gate"), scale=done.get("scale", 1.0), eps=eps, out=into,
                                          stream=stream)
                h = residual if pre is None else h
            if i < len(self.layers):
                y, done = self.forward_layer(i, h, stream=stream), lay
        if head is None:
            return residual, None if final_norm is None else h
        with _at(stream):
            if isinstance(head, torch.Tensor):
                return residual, linear_bf16(h, head)
            return residual, linear_int8(h, *head)

    def step(self, xs: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None,
             stream=None) -> List[torch.Tensor]:
        """One pass over the stack: layer i on xs[i] (the hidden state each layer receives;
        attention and the residual stream between layers are not part of this path)."""
        if len(xs) != len(self.layers):
            raise ValueError("one input per layer")
        res = []
        for i, x in enumerate(xs):
            res.append(self.forward_layer(i, x, None if outs is None else outs[i], stream=stream))
        return res


__all__ = ["plan_prefix", "cache_hits", "LayerStack"]
