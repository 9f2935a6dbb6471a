"""moe_linear over random sizes, types, forms, strides and offsets, one call after the other on buffers of their own: results
against 64 bits (the bounds of test_gpu_linear.py), and whatever lies around the rows of the output as it was."""
import math
import random

import pytest
import torch

import test_gpu_linear as plain
from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu


def _inside(t, unit, rng, fill):
    """The rows of t inside wider ones, at offsets that are multiples of `unit` elements, with a row before and one behind."""
    front = unit * rng.randint(0, 3)
    ld = (t.shape[1] + front + rng.randint(0, 24) + unit - 1) // unit * unit
    buf = torch.full((t.shape[0] + 2, ld), fill, dtype=t.dtype, device="cuda")
    view = buf[1:-1, front:front + t.shape[1]]
    view.copy_(t)
    return buf, view


@pytest.mark.parametrize("seed", range(4))
def test_random_calls(cuda_lib, seed):
    rng = random.Random(seed)
    spread = lambda low, high: int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    done = 0
    while done < 500:
        T, N, K = spread(1, 6000), spread(1, 9000), 8 * spread(1, 1024)
        if T * N * K > 2e10:
            continue
        done += 1
        dt, func, gated = rng.choice([torch.bfloat16, torch.float16]), rng.randrange(5), rng.random() < 0.4
        a = plain._make(T, N, K, dt, gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.6, seed=rng.randrange(1 << 30))
        ref, bound = plain._linear_ref(func=func, **a)
        if rng.random() < 0.6:
            a["x"] = _inside(a["x"], 8, rng, math.nan)[1]
            both = torch.cat([a["w"], a["w_mul"]]) if gated else a["w"]
            wide = _inside(both, 8, rng, math.nan)[1]  # one buffer: the same row stride
            a["w"], a["w_mul"] = wide[:N], wide[N:] if gated else None
        unit = rng.choice([1, 8])
        buf, out = _inside(torch.zeros(T, N, dtype=dt, device="cuda"), unit, rng, 7.0)
        if a["residual"] is not None:
            if rng.random() < 0.3:
                out.copy_(a["residual"])
                a["residual"] = out
            elif rng.random() < 0.5:
                a["residual"] = _inside(a["residual"], rng.choice([1, 2, 8]), rng, math.nan)[1]
        plain._run(a, func, out=out)
        plain._check(out, ref, bound, dt)
        around = buf.clone()
        around[1:-1].as_strided((T, N), (buf.stride(0), 1), out.storage_offset()).fill_(7.0)
        assert (around == 7.0).all(), f"written beside the rows: {T} x {N} x {K}"
