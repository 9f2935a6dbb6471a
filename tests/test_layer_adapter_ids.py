"""MoeLayer refuses adapter ids that moe_linear_adapters would refuse before it launches anything (CPU: every entry point that would
launch ends the test)."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi, layer as layer_module
from block_quantized_moe_router_gb300.layer import MoeLayer, _check_adapters

H, I, R, L = 64, 16, 8, 3


class _OnGpu(torch.Tensor):
    """A tensor that says it is on a GPU."""
    @property
    def is_cuda(self):
        return True


def _mk(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


@pytest.fixture
def layer(monkeypatch):
    def launched(*a, **kw):
        raise AssertionError("a kernel would have run")

    for name in ("moe_forward", "moe_ffn_forward", "moe_linear", "moe_linear_adapters", "moe_route", "moe_route_grouped", "moe_add_rms_norm",
                 "moe_sandwich_norm"):
        monkeypatch.setattr(layer_module.capi, name, launched)
    one = MoeLayer.__new__(MoeLayer)
    one.E, one.H, one.top_k, one.zero_experts, one.scoring, one.n_group = 4, H, 2, 0, capi.MOE_SCORE_SOFTMAX, 0
    one.norm_weight, one.norm_eps, one.post_norm_weight, one.block_gate, one.residual_scale, one.handle = _mk(H), 1e-6, None, None, 1.0, None
    one.shared = dict(gate=_mk(I, H), up=_mk(I, H), down=_mk(H, I), adapters=dict(gate_a=_mk(L, R, H), gate_b=_mk(L, I, R)))
    return one


BAD = [torch.zeros(5, dtype=torch.int64).as_subclass(_OnGpu), _mk(4, dtype=torch.int32), _mk(6, dtype=torch.int32), _mk(5, 1, dtype=torch.int32),
       _mk(10, dtype=torch.int32)[::2], torch.zeros(5, dtype=torch.int32), _mk(5, dtype=torch.float32)]


@pytest.mark.parametrize("ids", BAD, ids=[f"{tuple(t.shape)} {t.dtype}" for t in BAD])
@pytest.mark.parametrize("groups", [0, 2])
def test_refused_before_a_launch(layer, ids, groups):
    layer.n_group = groups
    x, out = _mk(5, H), torch.full((5, H), 7.0, dtype=torch.bfloat16)
    for call in (lambda: layer.forward(x, out=out, adapter_ids=ids), lambda: layer.ffn(x, _mk(5, 2, dtype=torch.int32), _mk(5, 2), out=out, adapter_ids=ids),
                 lambda: layer.block(x, adapter_ids=ids), lambda: layer.joined_block(x, x, adapter_ids=ids)):
        with pytest.raises(ValueError, match="adapter_ids"):
            call()
    assert (out == 7).all()


def test_adapters_off_16_bytes():
    """Nor does it take adapters that the kernels would refuse in every call."""
    s = dict(gate=_mk(I, H), up=_mk(I, H), down=_mk(H, I))
    good = dict(gate_a=_mk(L, R, H), gate_b=_mk(L, I, R), down_a=_mk(L, R, I), down_b=_mk(L, H, R))
    _check_adapters(good, s, H)
    for key, t in good.items():
        pool = _mk(t.numel() + 16)
        off = pool[1 if pool.data_ptr() % 16 == 0 else 0:][:t.numel()].view(t.shape)
        with pytest.raises(ValueError, match=key):
            _check_adapters({**good, key: off}, s, H)
    huge = dict(gate_a=_mk(1, 1, 1).expand((1 << 20) + 1, R, H), gate_b=good["gate_b"])
    with pytest.raises(ValueError, match="adapters"):
        _check_adapters(huge, s, H)
