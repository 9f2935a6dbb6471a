"""MoeLayer.block with hash routing, and what the layer refuses when it is built, on the GPU."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi, synth
from block_quantized_moe_router_gb300.layer import MoeLayer

pytestmark = pytest.mark.gpu


def _layer(cfg, inp, **kw):
    dev = lambda p: {k: (v.cuda().contiguous() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    opt = lambda key: inp[key].cuda().contiguous() if key in inp else None
    return MoeLayer(E=cfg.E, H=cfg.H, I=cfg.I, top_k=cfg.k, scoring=cfg.scoring, gate=dev(inp["gate"]), up=dev(inp["up"]),
                    down=dev(inp["down"]), w_router=opt("w_router"), correction_bias=opt("bias"), tid2eid=opt("tid2eid"),
                    renormalize=cfg.renorm, routed_scaling=cfg.scaling, act=cfg.act, **kw)


@pytest.mark.parametrize("scoring", [synth.SCORE_HASH, synth.SCORE_HASH_SQRTSOFTPLUS])
@pytest.mark.parametrize("T", [1, 40])
def test_hash_routed_block(cuda_lib, scoring, T):
    """The block is the norm and then the layer's forward, whatever routes it."""
    cfg = synth.MoeConfig("h", T=T, H=256, I=128, E=16, k=2, scoring=scoring, vocab=100)
    inp = synth.make_inputs(cfg, seed=T, device="cuda")
    weight = (1 + 0.1 * torch.randn(256, device="cuda")).bfloat16()
    layer = _layer(cfg, inp, norm_weight=weight)
    tokens = inp["token_ids"].cuda()
    delta, residual = (torch.randn(T, 256, device="cuda").bfloat16() for _ in range(2))
    out, r = layer.block(delta, residual, token_ids=tokens)
    n, s = torch.empty_like(delta), torch.empty_like(delta)
    capi.moe_add_rms_norm(delta, weight, n, residual=residual, sum_out=s)
    want = layer.forward(n, token_ids=tokens)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there, _ = layer.block(delta, residual, token_ids=tokens, stream=side)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    assert torch.equal(out, want) and torch.equal(r, s) and torch.equal(there, want)
    layer.close()


def test_shared_expert_is_checked_when_built(cuda_lib):
    cfg = synth.MoeConfig("c", T=2, H=256, I=128, E=8, k=2, scoring=synth.SCORE_SOFTMAX)
    inp = synth.make_inputs(cfg, seed=0, device="cuda")
    mk = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    good = dict(gate=mk(64, 256), up=mk(64, 256), down=mk(256, 64))
    for kw in (dict(gate=mk(64, 264)[:, 4:260]), dict(up=mk(64, 264)[:, :256]), dict(down=mk(256, 68)[:, :64]), dict(down=mk(64, 256).t()),
               dict(gate_bias=torch.zeros(63, device="cuda")), dict(down_bias=mk(256))):
        with pytest.raises(ValueError, match="shared"):
            _layer(cfg, inp, shared={**good, **kw})
    wide = dict(gate=mk(64, 264)[:, :256], up=mk(64, 264)[:, 8:], down=mk(256, 72)[:, 8:], gate_bias=torch.zeros(64, device="cuda"))
    layer = _layer(cfg, inp, shared=wide)
    x = inp["x"].cuda()
    assert torch.isfinite(layer.forward(x)[0].float()).all()
    layer.close()
