"""The distances that moe_linear_adapters passes on for its stacked adapters (CPU, plain memory in place of the device's)."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi

R, N, K = 8, 24, 40


def _pair(a, b):
    return capi._pair(a, b, torch.bfloat16, a.shape[0], R, N, K, -1, "")[2]


def test_stacks():
    pool_a, pool_b = torch.zeros(6, R, K + 8, dtype=torch.bfloat16), torch.zeros(6, N + 3, R, dtype=torch.bfloat16)
    a, b = pool_a[1::2, :, :K], pool_b[1::2, :N]
    assert _pair(a, b) == (K + 8, 2 * R * (K + 8), R, 2 * (N + 3) * R)


def test_a_lone_adapter_has_no_distance():
    """Whatever its view says: two matrices' lone adapters, cut out of pools of different shapes, go together."""
    one = torch.zeros(1, R, K, dtype=torch.bfloat16), torch.zeros(1, N, R, dtype=torch.bfloat16)
    cut = torch.zeros(R, 5, K, dtype=torch.bfloat16).transpose(0, 1)[2:3], torch.zeros(9, N, R, dtype=torch.bfloat16)[::4][1:2]
    far = torch.as_strided(one[0], (1, R, K), (0, K, 1)), torch.as_strided(one[1], (1, N, R), (1 << 40, R, 1))
    assert _pair(*one) == _pair(*far) == (K, R * K, R, N * R)
    assert _pair(cut[0], cut[1]) == (5 * K, R * 5 * K, R, N * R)


def test_refusals():
    a, b = torch.zeros(2, R, K, dtype=torch.bfloat16), torch.zeros(2, N, R, dtype=torch.bfloat16)
    for bad in ((a, None), (a.transpose(1, 2), b), (a.half(), b), (a, b[:1])):
        with pytest.raises(ValueError):
            _pair(*bad) if bad[1] is not None else capi._pair(a, None, torch.bfloat16, 2, R, N, K, -1, "")
