"""MoeLayer with adapters on its shared expert, and blocks joined by moe_sandwich_norm, on the GPU."""
import math

import pytest
import torch

from block_quantized_moe_router_gb300 import capi, synth
from block_quantized_moe_router_gb300.layer import MoeLayer

pytestmark = pytest.mark.gpu

H, I, R, L = 256, 192, 16, 5


def _shared(adapters=True, keys=("gate", "up", "down")):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    mk = lambda n, k: (r(n, k) / math.sqrt(k)).bfloat16()
    s = dict(gate=mk(I, H), up=mk(I, H), down=mk(H, I), gate_bias=0.1 * r(I))
    if adapters:
        ad = dict(scale=0.5 + torch.rand(L, generator=g, device="cuda"))
        for key, n, k in (("gate", I, H), ("up", I, H), ("down", H, I)):
            a, b = (r(L, R, k) / math.sqrt(k)).bfloat16(), (0.3 * r(L, n, R) / math.sqrt(R)).bfloat16()
            if key in keys:
                ad[key + "_a"], ad[key + "_b"] = a, b
        s["adapters"] = ad
    return s


def _layer(T, seed=0, groups=False, **kw):
    cfg = synth.MoeConfig("a", T=T, H=H, I=128, E=16, k=2, scoring=synth.SCORE_SOFTMAX)
    inp = synth.make_inputs(cfg, seed=seed, device="cuda")
    dev = lambda p: {k: (v.cuda().contiguous() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    if groups:
        kw.update(n_group=4, topk_group=2)
    return MoeLayer(E=cfg.E, H=H, I=cfg.I, top_k=cfg.k, scoring=cfg.scoring, gate=dev(inp["gate"]), up=dev(inp["up"]), down=dev(inp["down"]),
                    w_router=inp["w_router"].cuda(), renormalize=True, **kw), inp["x"].cuda()


def _ids(T):
    ids = (torch.arange(T, device="cuda") * 3 % (L + 1)).to(torch.int32)
    return torch.where(ids == L, -1, ids).to(torch.int32)


def _low(x, a, b, scale, ids):
    """The adapters' part in fp64."""
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64, device="cuda")
    for j in range(L):
        rows = ids == j
        out[rows] = float(scale[j]) * (x[rows].double() @ a[j].double().t()) @ b[j].double().t()
    return out


@pytest.mark.parametrize("T", [1, 6, 40, 300])
@pytest.mark.parametrize("groups", [False, True])
@pytest.mark.parametrize("keys", [("gate", "up", "down"), ("down",), ("gate",), ("up", "down")])
def test_shared_expert(cuda_lib, T, groups, keys):
    """The shared expert of the formula on top of the routed experts alone.  h is rounded once (2^-9 of each of its I
    products), the routed sum before it (2^-9 of itself), the result once more."""
    s = _shared(keys=keys)
    layer, x = _layer(T, groups=groups, shared=s)
    plain, _ = _layer(T, groups=groups)
    ids = _ids(T)
    out = layer.forward(x, adapter_ids=ids)[0]
    routed = plain.forward(x)[0]
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    ad = s["adapters"]
    low = lambda v, key: _low(v, ad[key + "_a"], ad[key + "_b"], ad["scale"], ids) if key in keys else 0
    z = x.double() @ s["gate"].double().t() + s["gate_bias"].double() + low(x, "gate")
    h = z * torch.sigmoid(z) * (x.double() @ s["up"].double().t() + low(x, "up"))
    want = h @ s["down"].double().t() + low(h, "down") + routed.double()
    size = h.abs() @ s["down"].double().abs().t() + routed.double().abs()
    if "down" in keys:
        for j in range(L):
            rows = ids == j
            size[rows] += float(ad["scale"][j]) * (h[rows].abs() @ ad["down_a"][j].double().abs().t()) @ ad["down_b"][j].double().abs().t()
    assert float(((out.double() - want).abs() - 2.0 ** -8 * size - 2.0 ** -9 * want.abs() - 1e-4).max()) <= 0
    # the routing and its outputs are those of the layer without adapters
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    assert not torch.equal(out, layer.forward(x, adapter_ids=none)[0]) or bool((ids < 0).all())
    ffn_ids, w, _ = layer.route(x)
    assert torch.equal(layer.ffn(x, ffn_ids, w, adapter_ids=ids), out) or not groups and T <= 8
    for la in (layer, plain):
        la.close()


def test_calls_without_ids_are_the_layer(cuda_lib):
    layer, x = _layer(40, shared=_shared())
    bare, _ = _layer(40, shared=_shared(adapters=False))
    assert torch.equal(layer.forward(x)[0], bare.forward(x)[0])
    with pytest.raises(ValueError, match="without adapters"):
        bare.forward(x, adapter_ids=_ids(40))
    alone, _ = _layer(40)
    with pytest.raises(ValueError, match="without adapters"):
        alone.forward(x, adapter_ids=_ids(40))
    bad = _ids(40)
    bad[3] = 77
    layer.forward(x, adapter_ids=bad)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == capi.MOE_DEV_BAD_ADAPTER_ID
    for la in (layer, bare, alone):
        la.close()


@pytest.mark.parametrize("T", [1, 7, 130])
@pytest.mark.parametrize("wide", [False, True])
def test_joined_blocks(cuda_lib, T, wide):
    """Three layers one after the other, each joined to the next: the calls of its parts, whatever stream and graph runs
    them."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = lambda: (0.1 * r(H)).bfloat16()
    layers = []
    for i in range(3):
        layer, x = _layer(T, seed=i, shared=_shared(), post_norm_weight=w(), block_gate=(0.5 + 0.1 * r(H)).bfloat16(), residual_scale=0.75,
                          norm_offset=1.0)
        layers.append(layer)
    pre = [w() for _ in range(3)] + [None]
    ids = _ids(T)
    stream_type = torch.float32 if wide else torch.bfloat16
    start = r(T, H).to(stream_type)
    rows = r(T)

    def chain(stream=None):
        res = start
        n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        s = torch.empty_like(start)
        x0 = start.bfloat16()
        capi.moe_sandwich_norm(x0, s, weight=pre[0], out=n, weight_offset=1.0, stream=stream)
        for i, layer in enumerate(layers):
            n, res = layer.joined_block(n, res, pre[i + 1], row_gate=rows, row_sigmoid=True, adapter_ids=ids, stream=stream)
        return n, res

    n, want = chain()
    assert n is None and want.dtype == stream_type
    # by parts
    res = start
    x0, s = start.bfloat16(), torch.empty_like(start)
    n = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    capi.moe_sandwich_norm(x0, s, weight=pre[0], out=n, weight_offset=1.0)
    for i, layer in enumerate(layers):
        y = layer.forward(n, adapter_ids=ids)[0]
        p = y.double() / (y.double().square().mean(1, keepdim=True) + 1e-6).sqrt() * (layer.post_norm_weight.double() + 1)
        q = 0.75 * res.double() + torch.sigmoid(rows.double())[:, None] * layer.block_gate.double() * p
        nxt, s = torch.empty_like(n), torch.empty_like(res)
        capi.moe_sandwich_norm(y, s, residual=res, post_weight=layer.post_norm_weight, gate=layer.block_gate, row_gate=rows, row_sigmoid=True,
                               weight=pre[i + 1], out=nxt if pre[i + 1] is not None else None, residual_scale=0.75, weight_offset=1.0)
        u = 2.0 ** -22 if wide else 2.0 ** -9
        assert float(((s.double() - q).abs() - 2.0 * u * q.abs() - 2e-5).max()) <= 0
        n, res = nxt, s
    assert torch.equal(res, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, there = chain(side)
    torch.cuda.synchronize()
    assert torch.equal(there, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, captured = chain()
    for _ in range(2):
        captured.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want)
    for layer in layers:
        assert int(layer.status.item()) == 0
        layer.close()
