"""moe_linear where the features end inside a warp's 32: lanes without one stay beside the others through the reads of
tensor memory (few rows, one part of K: no exchange), with a residual and without."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 16, 40, 100, 128, 200, 256])
@pytest.mark.parametrize("N", [7167, 7137, 4097, 2035, 1985, 300, 31, 1])
@pytest.mark.parametrize("K", [64, 256])
def test_features_that_end_inside_a_warp(cuda_lib, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    pick = lambda rows, cols: torch.randint(-1, 2, (rows, cols), generator=g, device="cuda").bfloat16()
    x, w, r = pick(T, K), pick(N, K), pick(T, N)
    # sums of whole numbers: exact in fp32, and below 257 exact in bf16
    want = x.double() @ w.double().t()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:-1]
    capi.moe_linear(x, w, out, dev_status=status)
    assert torch.equal(out.double(), want)
    capi.moe_linear(x, w, out, residual=r, dev_status=status)
    assert torch.equal(out.double(), want + r.double())
    assert int(status.item()) == 0 and (buf[0] == 7).all() and (buf[-1] == 7).all()
