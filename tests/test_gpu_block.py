"""The sublayer as a decoder runs it: residual add + RMS norm, routing over expert groups, FP4 experts,
bf16 shared expert, through MoeLayer -- against the oracle (experts) and plain 64-bit forms."""
import numpy as np
import pytest
import torch

import parity
from block_quantized_moe_router_gb300 import capi, synth
from block_quantized_moe_router_gb300.layer import MoeLayer

pytestmark = pytest.mark.gpu


def _layer(cfg, seed, shared_I=192, biases=True, **kw):
    inp = synth.make_inputs(cfg, seed=seed, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    shared = dict(gate=(r(shared_I, cfg.H) * 0.05).bfloat16(), up=(r(shared_I, cfg.H) * 0.05).bfloat16(),
                  down=(r(cfg.H, shared_I) * 0.05).bfloat16())
    if biases:
        shared.update(gate_bias=r(shared_I) * 0.1, up_bias=r(shared_I) * 0.1, down_bias=r(cfg.H) * 0.1)
    dev = lambda p: {k: (v.cuda().contiguous() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    layer = MoeLayer(E=cfg.E, H=cfg.H, I=cfg.I, top_k=cfg.k, scoring=cfg.scoring, gate=dev(inp["gate"]),
                     up=dev(inp["up"]), down=dev(inp["down"]), w_router=inp["w_router"].cuda(),
                     correction_bias=inp["bias"].cuda() if "bias" in inp else None, renormalize=cfg.renorm,
                     routed_scaling=cfg.scaling, act=cfg.act, shared=shared,
                     norm_weight=(1 + 0.1 * r(cfg.H)).bfloat16(), **kw)
    return layer, inp, shared


def _shared_ref(n, s):
    n = n.double()
    b = lambda key: s[key].double() if key in s else 0
    z = n @ s["gate"].double().t() + b("gate_bias")
    h = z * torch.sigmoid(z) * (n @ s["up"].double().t() + b("up_bias"))
    return h @ s["down"].double().t() + b("down_bias")


@pytest.mark.parametrize("T", [1, 5, 70, 300])
@pytest.mark.parametrize("act", [capi.MOE_ACT_BF16, capi.MOE_ACT_NVFP4])
def test_block(cuda_lib, T, act):
    cfg = synth.MoeConfig("b", T=T, H=512, I=256, E=24, k=4, scoring=synth.SCORE_SIGMOID, scaling=2.5, act=act)
    layer, inp, shared = _layer(cfg, seed=T, n_group=6, topk_group=3, group_top=2)
    delta = torch.randn(T, cfg.H, device="cuda").bfloat16()
    resid = (torch.randn(T, cfg.H, device="cuda") * 3).bfloat16()
    for residual in (resid, None):
        out, r = layer.block(delta, residual)
        torch.cuda.synchronize()
        assert int(layer.status.item()) == 0
        s = delta.double() + (0 if residual is None else residual.double())
        n64 = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * layer.norm_weight.double()
        # the norm's own rounding is checked here, what follows uses the rounded rows
        n, r2 = torch.empty_like(delta), torch.empty_like(delta)
        capi.moe_add_rms_norm(delta, layer.norm_weight, n, residual=residual, sum_out=r2, eps=1e-6)
        assert torch.equal(r, r2)
        assert float((n.double() - n64).norm()) <= 2 ** -8 * float(n64.norm())
        assert float((r.double() - s).norm()) <= 2 ** -8 * float(s.norm())
        ids, w, logits = layer.route(n)
        # the picks lie in the three best of the six groups
        v = torch.sigmoid(logits.double()) + layer.correction_bias.double()
        best = v.view(T, 6, 4).topk(2, 2).values.sum(2).topk(3, 1).indices
        assert ((ids // 4).unsqueeze(2) == best.unsqueeze(1)).any(2).all()
        ref = parity.oracle_ffn(cfg, dict(inp, x=n.cpu()), ids.cpu().numpy(), w.cpu().numpy().astype(np.float64))
        ref = ref + _shared_ref(n, shared).cpu().numpy()
        parity.assert_close(out, ref, "block")
        again, _ = layer.block(delta, residual)
        assert torch.equal(out, again)
    layer.close()


def test_shared_expert_without_groups(cuda_lib):
    """The bf16 shared expert joins every path of forward (one launch, many tokens)."""
    for T, act in ((3, capi.MOE_ACT_BF16), (40, capi.MOE_ACT_BF16), (140, capi.MOE_ACT_NVFP4)):
        cfg = synth.MoeConfig("s", T=T, H=512, I=256, E=16, k=2, scoring=synth.SCORE_SOFTMAX, act=act)
        layer, inp, shared = _layer(cfg, seed=T, biases=False)
        x = inp["x"].cuda()
        out, ids, w, _ = layer.forward(x)
        ref = parity.oracle_ffn(cfg, inp, ids.cpu().numpy(), w.cpu().numpy().astype(np.float64))
        parity.assert_close(out, ref + _shared_ref(x, shared).cpu().numpy())
        assert torch.equal(layer.ffn(x, ids, w), out)
        with pytest.raises(ValueError):
            layer.forward_host(inp["x"].cpu(), torch.empty(T, 512, dtype=torch.bfloat16))
        layer.close()


def test_block_in_a_graph(cuda_lib):
    cfg = synth.MoeConfig("g", T=4, H=512, I=256, E=24, k=4, scoring=synth.SCORE_SIGMOID)
    layer, inp, _ = _layer(cfg, seed=1, n_group=6, topk_group=2, group_top=1)
    a, b = (torch.randn(4, 512, device="cuda").bfloat16() for _ in range(2))
    want = [layer.block(t, inp["x"].cuda()) for t in (a, b)]
    x, res = a.clone(), inp["x"].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, r = layer.block(x, res)
    for t, (o, s) in ((b, want[1]), (a, want[0])):
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(r, s)
    layer.close()


def test_block_on_another_stream(cuda_lib):
    """What block() lets go of on its return is not handed out again while its stream still uses it."""
    cfg = synth.MoeConfig("t", T=300, H=512, I=256, E=24, k=4, scoring=synth.SCORE_SIGMOID, act=capi.MOE_ACT_BF16)
    layer, inp, shared = _layer(cfg, seed=3, n_group=6, topk_group=3, group_top=2)
    delta = torch.randn(300, 512, device="cuda").bfloat16()
    resid = torch.randn(300, 512, device="cuda").bfloat16()
    want = layer.block(delta, resid)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, mess = [], []
    for _ in range(30):
        got.append(layer.block(delta, resid, stream=side))
        mess.append([torch.full(shape, float("nan"), dtype=dt, device="cuda")  # on the current stream, at once
                     for shape, dt in (((300, 512), torch.bfloat16), ((300, 192), torch.bfloat16), ((300, 4), torch.float32),
                                       ((300, 24), torch.float32))])
        mess.pop()
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    for out, r in got:
        assert torch.equal(out, want[0]) and torch.equal(r, want[1])
    layer.close()


def test_streams_side_by_side(cuda_lib):
    """Every kind of kernel that waits within clusters, at once on streams of its own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    mk = lambda *s: (torch.randn(s, generator=g, device="cuda") / s[-1] ** 0.25).bfloat16()
    wg, wu, wd = mk(1024, 2048), mk(1024, 2048), mk(2048, 1024)
    jobs = []
    for T in (3, 128, 200, 700):  # one CTA per part of K, pairs, many rows
        x = mk(T, 2048)
        jobs.append(lambda o, x=x: capi.moe_linear(x, wg, o, w_mul=wu, func=capi.MOE_FUNC_SILU, stream=torch.cuda.current_stream()))
        jobs[-1].shape = (T, 1024)
        h = mk(T, 1024)
        jobs.append(lambda o, h=h: capi.moe_linear(h, wd, o, stream=torch.cuda.current_stream()))
        jobs[-1].shape = (T, 2048)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for T, E in ((40, 128), (500, 256), (300, 384)):
        x, w = mk(T, 2048), mk(E, 2048)
        logits, tw = torch.empty(T, E, device="cuda"), torch.empty(T, 6, device="cuda")
        jobs.append(lambda o, x=x, w=w, T=T, E=E, l=logits, tw=tw: capi.moe_route_grouped(
            T=T, E=E, H=2048, top_k=6, scoring=1, renormalize=True, routed_scaling=1.0, n_group=8, topk_group=3,
            group_top=2, x=x, w_router=w, logits_out=l, topk_ids=o, topk_w=tw, dev_status=status))
        jobs[-1].shape = (T, 6)
    kinds = [torch.int32 if j.shape[1] == 6 else torch.bfloat16 for j in jobs]
    want = [torch.empty(j.shape, dtype=t, device="cuda") for j, t in zip(jobs, kinds)]
    for j, o in zip(jobs, want):
        j(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[torch.empty_like(o) for _ in range(40)] for o in want]
    torch.cuda.synchronize()
    for i in range(40):
        for j, s, o in zip(jobs, streams, outs):
            with torch.cuda.stream(s):
                j(o[i])
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for o, w in zip(outs, want):
        assert all(torch.equal(t, w) for t in o)


def test_refusals(cuda_lib):
    cfg = synth.MoeConfig("r", T=2, H=256, I=128, E=8, k=2, scoring=synth.SCORE_SOFTMAX)
    with pytest.raises(ValueError):
        _layer(cfg, seed=0, n_group=4, topk_group=2, zero_experts=1)
    with pytest.raises(ValueError):
        _layer(cfg, seed=0, I_shared=128)
