"""MoeLayer: owns one layer's device buffers and calls the C ABI (marshalling only).

Weights are dicts of CUDA tensors ({packed, scales, globals, fmt}) laid out as include/moe.h
describes.  The layer prepares them once (moe_prepare_weights), keeps a workspace sized for
the largest token count seen, and runs route + FFN on the current CUDA stream with no host
synchronisation.

Optional parts around the expert FFN:
  n_group / topk_group / group_top   routing limited to expert groups (moe_route_grouped)
  shared   a bf16 shared expert {gate, up [I][H], down [H][I], and float biases gate_bias, up_bias
           [I], down_bias [H] if it has them}, added through moe_linear; instead of an FP4 one.
           It is added to the routed experts' sum as that was rounded to bf16, and the result is
           rounded again; an FP4 shared expert joins the sum in fp32
  shared["adapters"]   low-rank adapters of many requests on the shared expert (moe_linear_adapters):
           {gate_a, up_a [L][R][H], gate_b, up_b [L][I][R], down_a [L][R][I], down_b [L][H][R]}, each pair
           or not, all of one rank, and a float scale [L]; calls name each row's adapter in adapter_ids
  norm_weight / norm_eps   the RMS norm before the layer, with the residual add (block())
  post_norm_weight / block_gate / residual_scale / norm_offset   the norm behind the layer, its gate per
           channel, the scale of the residual and what is added to the norms' weights (joined_block())
"""
from __future__ import annotations

from typing import Optional

import torch

from . import capi


def _check_groups(E, top_k, scoring, zero_experts, n_group, topk_group, group_top):
    """The rules of moe_route_grouped that do not depend on a call."""
    if zero_experts or scoring in (capi.MOE_SCORE_HASH, capi.MOE_SCORE_HASH_SQRTSOFTPLUS):
        raise ValueError("expert groups need a learned router without zero-computation experts")
    if not 1 <= n_group <= 64 or E % n_group:
        raise ValueError(f"n_group must be 1 to 64 and divide the {E} experts, got {n_group}")
    if not 1 <= topk_group <= n_group:
        raise ValueError(f"topk_group must be 1 to n_group ({n_group}), got {topk_group}")
    size = E // n_group
    if group_top not in (1, 2) or group_top > size:
        raise ValueError(f"group_top must be 1 or 2 and at most the {size} experts of a group, got {group_top}")
    if top_k > topk_group * size:
        raise ValueError(f"top_k {top_k} exceeds the {topk_group * size} experts of {topk_group} groups")


def _check_shared(s, H):
    """The rules of moe_linear for the two products of the bf16 shared expert, before any kernel runs."""
    missing = [key for key in ("gate", "up", "down") if s.get(key) is None]
    if missing:
        raise ValueError(f"the shared expert needs gate, up and down; {missing[0]} is missing")
    I = s["gate"].shape[0]
    if I < 8 or I % 8:
        raise ValueError(f"the shared expert's width must be a multiple of 8, got {I}")
    for key, shape in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        t = s[key]
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_cuda:
            raise ValueError(f"shared {key} must be a bfloat16 CUDA matrix {shape}, got {t.dtype} {tuple(t.shape)} on {t.device}")
        if t.stride(1) != 1 or t.stride(0) % 8 or t.stride(0) < shape[1] or t.data_ptr() % 16:
            raise ValueError(f"shared {key} must have contiguous rows that start at multiples of 16 bytes")
    if s["up"].stride(0) != s["gate"].stride(0):
        raise ValueError("shared up must have the row stride of gate")
    for key, n in (("gate_bias", I), ("up_bias", I), ("down_bias", H)):
        t = s.get(key)
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (n,) or not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"shared {key} must be a contiguous float32 CUDA tensor ({n},), got {t.dtype} {tuple(t.shape)} on {t.device}")


def _check_adapters(ad, s, H):
    """The rules of moe_linear_adapters for the shared expert's adapters, before any kernel runs."""
    I = s["gate"].shape[0]
    sizes = None
    for key, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
        a, b = ad.get(key + "_a"), ad.get(key + "_b")
        if (a is None) != (b is None):
            raise ValueError(f"adapters of {key} need {key}_a and {key}_b")
        if a is None:
            continue
        if sizes is None:
            sizes = tuple(a.shape[:2])
            if len(sizes) < 2 or not 1 <= sizes[0] <= 1 << 20 or sizes[1] % 8 or not 8 <= sizes[1] <= 256:
                raise ValueError(f"adapters need ranks that are multiples of 8 up to 256, at most 2^20 of them, got {key}_a {tuple(a.shape)}")
        for name, t, shape in ((key + "_a", a, sizes + (cols,)), (key + "_b", b, (sizes[0], rows, sizes[1]))):
            if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor {shape}, got {t.dtype} {tuple(t.shape)} on {t.device}")
            if t.data_ptr() % 16:
                raise ValueError(f"{name} of the adapters must start at a multiple of 16 bytes")
    if sizes is None:
        raise ValueError("adapters hold none of gate, up and down")
    scale = ad.get("scale")
    if scale is not None and (scale.dtype != torch.float32 or tuple(scale.shape) != sizes[:1] or not scale.is_cuda or not scale.is_contiguous()):
        raise ValueError(f"adapters' scale must be a contiguous float32 CUDA tensor {sizes[:1]}, got {scale.dtype} {tuple(scale.shape)} on {scale.device}")


class MoeLayer:
    def __init__(self, *, E, H, I, top_k, scoring, gate, up, down, I_shared=0, sh_gate=None,
                 sh_up=None, sh_down=None, w_router=None, correction_bias=None, tid2eid=None,
                 renormalize=True, routed_scaling=1.0, act=capi.MOE_ACT_BF16, g_act1=1.0,
                 g_act2=1.0, zero_experts=0, n_group=0, topk_group=0, group_top=2, shared=None,
                 norm_weight=None, norm_eps=1e-6, post_norm_weight=None, block_gate=None,
                 residual_scale=1.0, norm_offset=0.0):
        self.E, self.H, self.I, self.top_k, self.I_shared = E, H, I, top_k, I_shared
        self.zero_experts = zero_experts
        self.scoring, self.renormalize, self.routed_scaling = scoring, renormalize, routed_scaling
        self.act, self.g_act1, self.g_act2 = act, g_act1, g_act2
        self.w_router, self.correction_bias, self.tid2eid = w_router, correction_bias, tid2eid
        if n_group:
            _check_groups(E, top_k, scoring, zero_experts, n_group, topk_group, group_top)
        if shared is not None:
            if I_shared:
                raise ValueError("a layer has one shared expert: FP4 (I_shared) or bf16 (shared)")
            _check_shared(shared, H)
            if shared.get("adapters") is not None:
                _check_adapters(shared["adapters"], shared, H)
        for name, w in (("norm_weight", norm_weight), ("post_norm_weight", post_norm_weight), ("block_gate", block_gate)):
            if w is not None and (w.dtype != torch.bfloat16 or tuple(w.shape) != (H,)):
                raise ValueError(f"{name} must be a bfloat16 tensor ({H},), got {w.dtype} {tuple(w.shape)}")
        if norm_weight is not None and norm_offset:
            raise ValueError("norm_offset belongs to joined_block, whose caller norms the first rows; a layer with norm_weight has none")
        self.n_group, self.topk_group, self.group_top = n_group, topk_group, group_top
        self.shared, self.norm_weight, self.norm_eps = shared, norm_weight, norm_eps
        self.post_norm_weight, self.block_gate = post_norm_weight, block_gate
        self.residual_scale, self.norm_offset = residual_scale, norm_offset
        self._weights = (gate, up, down, sh_gate, sh_up, sh_down)  # keep alive
        self.desc = capi.ffn_desc(E, H, I, top_k, I_shared, gate, up, down, sh_gate, sh_up, sh_down,
                                  zero_experts)
        self.handle = capi.moe_prepare_weights(self.desc)
        self._ws = None
        self._ws_host = None
        self._ws_adapters = None
        self._outgrown = []
        self._host_route = {}
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    @classmethod
    def from_inputs(cls, inp: dict, device="cuda"):
        """Build from a synth.make_inputs() dict (tensors moved to `device`)."""
        cfg = inp["cfg"]

        def dev(p):
            if p is None:
                return None
            return {k: (v.to(device).contiguous() if isinstance(v, torch.Tensor) else v)
                    for k, v in p.items()}

        opt = lambda key: inp[key].to(device).contiguous() if key in inp else None
        return cls(E=cfg.E, H=cfg.H, I=cfg.I, top_k=cfg.k, scoring=cfg.scoring,
                   gate=dev(inp["gate"]), up=dev(inp["up"]), down=dev(inp["down"]),
                   I_shared=cfg.I_shared, sh_gate=dev(inp.get("sh_gate")),
                   sh_up=dev(inp.get("sh_up")), sh_down=dev(inp.get("sh_down")),
                   w_router=opt("w_router"), correction_bias=opt("bias"), tid2eid=opt("tid2eid"),
                   renormalize=cfg.renorm, routed_scaling=cfg.scaling, act=cfg.act,
                   zero_experts=cfg.zero_experts)

    def close(self):
        if self.handle:
            capi.moe_release_weights(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, T: int, stream=None) -> torch.Tensor:
        """Scratch memory for T tokens, for work on `stream` (the current one by default).  One call of a layer uses it at a
        time: calls on several streams have to wait for one another."""
        self._ws = self._grown(self._ws, capi.moe_workspace_size(self.desc, T, self.act), stream)
        return self._ws

    def _grown(self, ws, need, stream=None):
        """`ws`, or a larger one in its place.  The one that was outgrown stays with the layer: a captured graph keeps
        its address, another stream may still be using it.  Steps of half of it at least bound the sum of them all.
        The new one comes from the pool of the stream that uses it: memory that another stream's pool hands out may
        still be in use by work queued there."""
        if ws is not None and ws.numel() >= need:
            return ws
        size = max(need, 256)
        if ws is not None:
            self._outgrown.append(ws)
            size = max(size, ws.numel() + ws.numel() // 2)
        if stream is None:
            return torch.empty(size, dtype=torch.uint8, device="cuda")
        with torch.cuda.stream(stream):
            return torch.empty(size, dtype=torch.uint8, device="cuda")

    def route(self, x=None, *, token_ids=None, logits_in=None, topk_ids=None, topk_w=None,
              logits_out=None, stream=None):
        T = (x.shape[0] if x is not None else
             token_ids.shape[0] if token_ids is not None else logits_in.shape[0])
        if topk_ids is None:
            topk_ids = torch.empty((T, self.top_k), dtype=torch.int32, device="cuda")
        if topk_w is None:
            topk_w = torch.empty((T, self.top_k), dtype=torch.float32, device="cuda")
        if (logits_out is None and logits_in is None and self.scoring != capi.MOE_SCORE_HASH):
            logits_out = torch.empty((T, self.E + self.zero_experts), dtype=torch.float32,
                                     device="cuda")
        if self.n_group:
            capi.moe_route_grouped(T=T, E=self.E, H=self.H, top_k=self.top_k, scoring=self.scoring,
                                   renormalize=self.renormalize, routed_scaling=self.routed_scaling,
                                   n_group=self.n_group, topk_group=self.topk_group,
                                   group_top=self.group_top, x=x, w_router=self.w_router,
                                   logits_in=logits_in, logits_out=logits_out,
                                   correction_bias=self.correction_bias, topk_ids=topk_ids,
                                   topk_w=topk_w, dev_status=self.status, stream=stream)
            return topk_ids, topk_w, logits_out
        capi.moe_route(T=T, E=self.E, H=self.H, top_k=self.top_k, scoring=self.scoring,
                       renormalize=self.renormalize, routed_scaling=self.routed_scaling, x=x,
                       w_router=None if logits_in is not None else self.w_router,
                       logits_in=logits_in, logits_out=logits_out,
                       correction_bias=self.correction_bias, tid2eid=self.tid2eid,
                       vocab=0 if self.tid2eid is None else self.tid2eid.shape[0],
                       token_ids=token_ids, topk_ids=topk_ids, topk_w=topk_w,
                       dev_status=self.status, stream=stream, zero_experts=self.zero_experts)
        return topk_ids, topk_w, logits_out

    def ffn(self, x, topk_ids, topk_w, out=None, stream=None, adapter_ids=None):
        ad = self._adapters(adapter_ids, x)
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.bfloat16, device="cuda")
        capi.moe_ffn_forward(self.handle, T, self.act, self.g_act1, self.g_act2, x, topk_ids,
                             topk_w, out, self.workspace(T, stream), dev_status=self.status, stream=stream)
        self._add_shared(x, out, stream, ad, adapter_ids)
        return out

    def _add_shared(self, x, out, stream, ad=None, adapter_ids=None):
        """out += down(SiLU(gate x) * up x) of the bf16 shared expert, if the layer has one."""
        if self.shared is None:
            return
        s = self.shared
        T, I = x.shape[0], s["gate"].shape[0]
        with torch.cuda.stream(stream):  # h is freed before it is used up: only that stream may have it next
            h = torch.empty((T, I), dtype=torch.bfloat16, device="cuda")
        self._linear(ad, "gate", "up", adapter_ids, x, s["gate"], h, w_mul=s["up"], bias=s.get("gate_bias"),
                     bias_mul=s.get("up_bias"), func=capi.MOE_FUNC_SILU, stream=stream)
        self._linear(ad, "down", None, adapter_ids, h, s["down"], out, bias=s.get("down_bias"), residual=out,
                     stream=stream)

    def _adapters(self, adapter_ids, x):
        """The shared expert's adapters for a call that names them for the rows of x, None for one that does not.  What is wrong
        with the ids is said here, before a kernel has written anything."""
        if adapter_ids is None:
            return None
        ad = None if self.shared is None else self.shared.get("adapters")
        if ad is None:
            raise ValueError("the layer was built without adapters")
        if (adapter_ids.dtype != torch.int32 or adapter_ids.shape != x.shape[:1] or not adapter_ids.is_cuda
                or not adapter_ids.is_contiguous() or adapter_ids.get_device() != x.get_device()):
            raise ValueError(f"adapter_ids must be a contiguous int32 tensor {tuple(x.shape[:1])} on the device of x, "
                             f"got {adapter_ids.dtype} {tuple(adapter_ids.shape)} on {adapter_ids.device}")
        return ad

    def _linear(self, ad, key, mul, ids, x, w, out, **kw):
        """moe_linear of the shared expert, with the adapters of `key` (and `mul`) where there are some."""
        pairs = {} if ad is None else {"a": ad.get(key + "_a"), "b": ad.get(key + "_b")}
        if ad is not None and mul is not None:
            pairs.update(a_mul=ad.get(mul + "_a"), b_mul=ad.get(mul + "_b"))
        given = [t for t in (pairs.get("a"), pairs.get("a_mul")) if t is not None]
        if not given:
            return capi.moe_linear(x, w, out, dev_status=self.status, **kw)
        self._ws_adapters = self._grown(self._ws_adapters,
                                        capi.moe_adapter_workspace_size(x.shape[0], given[0].shape[1], len(given)),
                                        kw.get("stream"))
        capi.moe_linear_adapters(x, w, out, ids, scale=ad.get("scale"), workspace=self._ws_adapters,
                                 dev_status=self.status, **pairs, **kw)

    def block(self, delta, residual=None, *, token_ids=None, logits_in=None, adapter_ids=None, stream=None):
        """The layer with the residual add and norm before it: r = delta + residual, n = RMS norm of
        r, and (FFN of n, r), the next layer's delta and residual.  Without a residual r = delta.
        token_ids: of the rows, for hash routing.  The results belong to `stream` (the current one
        by default)."""
        if self.norm_weight is None:
            raise ValueError("the layer was built without norm_weight")
        if self.post_norm_weight is not None or self.block_gate is not None or self.residual_scale != 1:
            raise ValueError("block() has no norm behind the layer, no gate and no residual scale; joined_block() has")
        if stream is not None:  # what is freed on return goes back to the stream that still uses it
            with torch.cuda.stream(stream):
                return self.block(delta, residual, token_ids=token_ids, logits_in=logits_in, adapter_ids=adapter_ids)
        self._adapters(adapter_ids, delta)
        n = torch.empty_like(delta)
        r = torch.empty_like(delta)
        capi.moe_add_rms_norm(delta, self.norm_weight, n, residual=residual, sum_out=r,
                              eps=self.norm_eps)
        return self.forward(n, token_ids=token_ids, logits_in=logits_in, adapter_ids=adapter_ids)[0], r

    def joined_block(self, n, residual, next_weight=None, *, row_gate=None, row_sigmoid=False, token_ids=None,
                     logits_in=None, adapter_ids=None, stream=None):
        """The layer on rows n that are normed already, and what stands between it and the next block in one pass
        (moe_sandwich_norm): the norm behind it (post_norm_weight), its gates, the residual add and, with next_weight,
        the norm before the next block.  residual is bf16 or float32 and stays so.  Returns (the next block's n or
        None, its residual).  The results belong to `stream` (the current one by default)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.joined_block(n, residual, next_weight, row_gate=row_gate, row_sigmoid=row_sigmoid,
                                         token_ids=token_ids, logits_in=logits_in, adapter_ids=adapter_ids)
        y = self.forward(n, token_ids=token_ids, logits_in=logits_in, adapter_ids=adapter_ids)[0]
        s = torch.empty(residual.shape, dtype=residual.dtype, device=residual.device)
        out = None if next_weight is None else y
        capi.moe_sandwich_norm(y, s, residual=residual, post_weight=self.post_norm_weight, gate=self.block_gate,
                               row_gate=row_gate, row_sigmoid=row_sigmoid, weight=next_weight, out=out,
                               residual_scale=self.residual_scale, weight_offset=self.norm_offset, eps=self.norm_eps)
        return out, s

    def forward(self, x=None, *, token_ids=None, logits_in=None, out=None, topk_ids=None,
                topk_w=None, logits_out=None, adapter_ids=None, stream=None):
        """Route + FFN through moe_forward (one launch for a few tokens; with expert groups the
        routing runs first on its own).  adapter_ids: int32, each row's adapter of the shared expert, -1
        for none.  Returns (out, topk_ids, topk_w, logits_out)."""
        ad = self._adapters(adapter_ids, x)
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.bfloat16, device="cuda")
        if self.n_group:
            topk_ids, topk_w, logits_out = self.route(
                x, logits_in=logits_in, topk_ids=topk_ids, topk_w=topk_w, logits_out=logits_out,
                stream=stream)
            return self.ffn(x, topk_ids, topk_w, out=out, stream=stream, adapter_ids=adapter_ids), topk_ids, topk_w, logits_out
        if topk_ids is None:
            topk_ids = torch.empty((T, self.top_k), dtype=torch.int32, device="cuda")
        if topk_w is None:
            topk_w = torch.empty((T, self.top_k), dtype=torch.float32, device="cuda")
        if (logits_out is None and logits_in is None and self.scoring != capi.MOE_SCORE_HASH):
            logits_out = torch.empty((T, self.E + self.zero_experts), dtype=torch.float32,
                                     device="cuda")
        d = capi.route_desc(T=T, E=self.E, H=self.H, top_k=self.top_k, scoring=self.scoring,
                            renormalize=self.renormalize, routed_scaling=self.routed_scaling,
                            w_router=None if logits_in is not None else self.w_router,
                            correction_bias=self.correction_bias, tid2eid=self.tid2eid,
                            vocab=0 if self.tid2eid is None else self.tid2eid.shape[0],
                            token_ids=token_ids, zero_experts=self.zero_experts)
        capi.moe_forward(self.handle, d, self.act, self.g_act1, self.g_act2, x, topk_ids, topk_w,
                         out, self.workspace(T, stream), logits_in=logits_in, logits_out=logits_out,
                         dev_status=self.status, stream=stream)
        self._add_shared(x, out, stream, ad, adapter_ids)
        return out, topk_ids, topk_w, logits_out

    def forward_host(self, x_host, out_host, *, token_ids_host=None, topk_ids_host=None,
                     topk_w_host=None, stream=None):
        """Route + FFN on host buffers through moe_forward_host: x_host (and token_ids_host for
        hash routing) are copied in, out_host (and the ids / weights when given) copied back, all
        enqueued on the stream; the caller synchronises before reading the outputs."""
        if self.n_group or self.shared is not None:
            raise ValueError("the host-buffer entry has no expert groups and no bf16 shared expert")
        T = x_host.shape[0]
        cached = self._host_route.get(T)
        if cached is None:
            d = capi.route_desc(T=T, E=self.E, H=self.H, top_k=self.top_k, scoring=self.scoring,
                                renormalize=self.renormalize, routed_scaling=self.routed_scaling,
                                w_router=self.w_router, correction_bias=self.correction_bias,
                                tid2eid=self.tid2eid,
                                vocab=0 if self.tid2eid is None else self.tid2eid.shape[0],
                                zero_experts=self.zero_experts)
            cached = self._host_route[T] = (d, capi.moe_workspace_size_host(self.desc, T, self.act))
        d, need = cached
        self._ws_host = self._grown(self._ws_host, need, stream)
        capi.moe_forward_host(self.handle, d, self.act, self.g_act1, self.g_act2, x_host, out_host,
                              self._ws_host, token_ids_host=token_ids_host,
                              topk_ids_host=topk_ids_host, topk_w_host=topk_w_host,
                              dev_status=self.status, stream=stream)
        return out_host
