"""MoeLayer refuses expert groups, a shared expert or a norm weight that no call could use when it is built, before it
prepares weights (CPU)."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi
from block_quantized_moe_router_gb300.layer import MoeLayer


def _build(**kw):
    args = dict(E=24, H=256, I=128, top_k=4, scoring=capi.MOE_SCORE_SIGMOID, gate=None, up=None, down=None)
    return MoeLayer(**{**args, **kw})


@pytest.mark.parametrize("kw", [dict(n_group=6), dict(n_group=6, topk_group=7), dict(n_group=5, topk_group=2), dict(n_group=6, topk_group=-1),
                                dict(n_group=-6, topk_group=1), dict(n_group=65, topk_group=3, E=130), dict(n_group=6, topk_group=2, group_top=3),
                                dict(n_group=6, topk_group=2, group_top=0), dict(n_group=24, topk_group=5), dict(n_group=12, topk_group=1),
                                dict(n_group=6, topk_group=2, zero_experts=1), dict(n_group=6, topk_group=2, scoring=capi.MOE_SCORE_HASH)])
def test_groups(kw):
    with pytest.raises(ValueError, match="group|top_k"):
        _build(**kw)


def _shared(I=64, H=256, device="meta", **kw):
    t = dict(gate=torch.empty(I, H, dtype=torch.bfloat16, device=device), up=torch.empty(I, H, dtype=torch.bfloat16, device=device),
             down=torch.empty(H, I, dtype=torch.bfloat16, device=device))
    return {**t, **kw}


def test_shared_expert():
    for shared in (_shared(H=128), _shared(I=60), _shared(up=None), _shared(device="cpu"), _shared(gate=torch.empty(64, 256)),
                   _shared(down=torch.empty(64, 256, dtype=torch.bfloat16)), {}):
        with pytest.raises(ValueError, match="shared"):
            _build(shared=shared)
    with pytest.raises(ValueError, match="one shared expert"):
        _build(shared=_shared(), I_shared=128)


def test_norm_weight():
    for w in (torch.ones(255, dtype=torch.bfloat16), torch.ones(256)):
        with pytest.raises(ValueError, match="norm_weight"):
            _build(norm_weight=w)
