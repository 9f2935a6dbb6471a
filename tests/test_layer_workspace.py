"""MoeLayer's workspaces outlive their replacement: a captured graph, or a stream that still runs, may use the one that a longer
call has outgrown (CPU, with plain memory in place of the device's)."""
import types
import weakref

import torch

from block_quantized_moe_router_gb300 import layer as layer_module
from block_quantized_moe_router_gb300.layer import MoeLayer


def _layer(monkeypatch, sizes):
    monkeypatch.setattr(layer_module.capi, "moe_workspace_size", lambda desc, T, act: sizes(T))
    fake = types.SimpleNamespace(empty=lambda *a, device=None, **kw: torch.empty(*a, **kw), uint8=torch.uint8)
    monkeypatch.setattr(layer_module, "torch", fake)
    one = MoeLayer.__new__(MoeLayer)
    one.desc, one.act, one.handle = None, 0, None
    one._ws = one._ws_host = None
    one._outgrown = []
    return one


def test_an_outgrown_workspace_stays(monkeypatch):
    one = _layer(monkeypatch, lambda T: 1000 * T)
    first = weakref.ref(one.workspace(4))
    second = weakref.ref(one.workspace(300))
    assert second().numel() >= 300000 and first() is not None and first().numel() >= 4000
    assert one.workspace(5) is second()
    one = None
    assert first() is None and second() is None  # with the layer they go


def test_growth_by_small_steps_stays_bounded(monkeypatch):
    one = _layer(monkeypatch, lambda T: 1000 * T)
    for T in range(1, 2000):
        assert one.workspace(T).numel() >= 1000 * T
    held = one._ws.numel() + sum(w.numel() for w in one._outgrown)
    assert held <= 4.5 * 1000 * 2000  # at most half beyond the need, and twice that in all that came before
