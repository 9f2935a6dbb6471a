"""A layer built with what stands behind it (a norm, a gate, a residual scale) is not run by the call that knows none of them (CPU)."""
import pytest
import torch

from block_quantized_moe_router_gb300 import layer as layer_module
from block_quantized_moe_router_gb300.layer import MoeLayer

H = 64


def _layer(**kw):
    one = MoeLayer.__new__(MoeLayer)
    one.H, one.handle, one.shared = H, None, None
    one.norm_weight, one.norm_eps, one.norm_offset = torch.ones(H, dtype=torch.bfloat16), 1e-6, 0.0
    one.post_norm_weight, one.block_gate, one.residual_scale = None, None, 1.0
    for name, value in kw.items():
        setattr(one, name, value)
    return one


@pytest.mark.parametrize("kw", [dict(post_norm_weight=torch.ones(H, dtype=torch.bfloat16)), dict(block_gate=torch.ones(H, dtype=torch.bfloat16)),
                                dict(residual_scale=0.5)])
def test_block_refuses(monkeypatch, kw):
    monkeypatch.setattr(layer_module.capi, "moe_add_rms_norm", lambda *a, **k: pytest.fail("a kernel would have run"))
    with pytest.raises(ValueError, match="joined_block"):
        _layer(**kw).block(torch.zeros(3, H, dtype=torch.bfloat16))


def test_block_of_a_plain_layer(monkeypatch):
    monkeypatch.setattr(layer_module.capi, "moe_add_rms_norm", lambda *a, **k: None)
    one = _layer()
    one.forward = lambda n, **kw: ("out",)
    assert one.block(torch.zeros(3, H, dtype=torch.bfloat16))[0] == "out"
