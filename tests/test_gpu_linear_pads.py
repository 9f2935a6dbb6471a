"""moe_linear with many rows that start at multiples of 16 bytes and end inside 16: what lies behind a row stays as it was."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [(3000, 2047, 64), (2500, 1001, 136), (1007, 2965, 24), (4704, 85, 672), (2869, 580, 400),
                                   (5987, 650, 72), (2049, 1156, 64), (4452, 162, 1016), (600, 7169, 128), (3000, 2048, 64)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_inside_wider_ones(cuda_lib, T, N, K, gated, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    pick = lambda rows, cols: torch.randint(-1, 2, (rows, cols), generator=g, device="cuda").to(dtype)
    # sums of whole numbers are exact in fp32; their product (an integer below 2^24) is rounded once, like the sum
    x, w, v = pick(T, K), pick(N, K), pick(N, K) if gated else None
    want = x.float() @ w.float().t()
    if gated:
        want = want * (x.float() @ v.float().t())
    ld = (N + 7) // 8 * 8 + 16
    for residual in (False, True):
        buf = torch.full((T + 2, ld), 7.0, dtype=dtype, device="cuda")
        out = buf[1:-1, 8:8 + N]
        res = None
        if residual:
            res = torch.full((T + 2, ld), 5.0, dtype=dtype, device="cuda")[1:-1, 8:8 + N]
            res.copy_(pick(T, N))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        capi.moe_linear(x, w, out, w_mul=v, residual=res, dev_status=status)
        assert int(status.item()) == 0
        assert torch.equal(out, (want + (res.float() if residual else 0)).to(dtype))
        rest = buf.clone()
        rest[1:-1, 8:8 + N] = 7.0
        assert (rest == 7.0).all()
