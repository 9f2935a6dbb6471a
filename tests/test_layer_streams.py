"""MoeLayer's workspaces come from the pool of the stream that uses them (CPU, with plain memory in place of the device's).  The
current stream's pool hands out memory that work queued there may still be using, and another stream does not wait for that work."""
import contextlib
import types

import pytest
import torch

from block_quantized_moe_router_gb300 import layer as layer_module
from block_quantized_moe_router_gb300.layer import MoeLayer


@pytest.fixture
def layer(monkeypatch):
    """A layer without kernels, and the stream of each allocation of bytes."""
    made, current = [], ["current"]

    @contextlib.contextmanager
    def stream(s):
        before = current[0]
        current[0] = before if s is None else s
        yield
        current[0] = before

    def empty(*a, device=None, dtype=None):
        if dtype is torch.uint8:
            made.append(current[0])
        return torch.empty(*a, dtype=dtype)

    nothing = lambda *a, **kw: None
    for name in ("moe_forward", "moe_ffn_forward", "moe_linear", "moe_linear_adapters", "moe_forward_host"):
        monkeypatch.setattr(layer_module.capi, name, nothing)
    monkeypatch.setattr(layer_module.capi, "route_desc", nothing)
    monkeypatch.setattr(layer_module.capi, "moe_workspace_size", lambda desc, T, act: 1000 * T)
    monkeypatch.setattr(layer_module.capi, "moe_workspace_size_host", lambda desc, T, act: 1000 * T)
    monkeypatch.setattr(layer_module.capi, "moe_adapter_workspace_size", lambda T, R, matrices: 100 * T * R * matrices)
    fake = types.SimpleNamespace(empty=empty, uint8=torch.uint8, bfloat16=torch.bfloat16, float32=torch.float32, int32=torch.int32,
                                 cuda=types.SimpleNamespace(stream=stream))
    monkeypatch.setattr(layer_module, "torch", fake)
    one = MoeLayer.__new__(MoeLayer)
    one.E, one.H, one.top_k, one.zero_experts, one.scoring, one.n_group = 4, 64, 2, 0, 0, 0
    one.act = one.g_act1 = one.g_act2 = one.routed_scaling = 0
    one.renormalize, one.w_router, one.correction_bias, one.tid2eid = True, None, None, None
    one.desc = one.handle = one.status = one._ws = one._ws_host = one._ws_adapters = None
    one._outgrown, one._host_route = [], {}
    mk = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    one.shared = dict(gate=mk(16, 64), up=mk(16, 64), down=mk(64, 16), adapters=dict(
        gate_a=mk(3, 8, 64), gate_b=mk(3, 16, 8), down_a=mk(3, 8, 16), down_b=mk(3, 64, 8)))
    return one, made


class _OnGpu(torch.Tensor):
    """A tensor that says it is on a GPU."""
    @property
    def is_cuda(self):
        return True


def _ids(T):
    return torch.zeros(T, dtype=torch.int32).as_subclass(_OnGpu)


def test_forward_and_adapters(layer):
    one, made = layer
    x = torch.zeros(5, 64, dtype=torch.bfloat16)
    one.forward(x, adapter_ids=_ids(5), stream="side")
    assert made == ["side", "side"]  # the experts', the adapters'
    one.forward(x, adapter_ids=_ids(5), stream="side")
    assert len(made) == 2
    one.forward(torch.zeros(50, 64, dtype=torch.bfloat16), adapter_ids=_ids(50))
    assert made[2:] == ["current", "current"]


def test_ffn_and_host(layer):
    one, made = layer
    x = torch.zeros(5, 64, dtype=torch.bfloat16)
    one.ffn(x, None, None, adapter_ids=_ids(5), stream="side")
    assert made == ["side", "side"]
    one.shared = None
    one.forward_host(x, x, stream="other")
    assert made[2:] == ["other"]
