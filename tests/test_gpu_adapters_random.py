"""moe_linear_adapters at drawn sizes, strides, ids and forms, call after call without a synchronisation between."""
import random

import pytest
import torch

from test_gpu_adapters import DT, _check, _make, _reference, _workspace
from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu


def _draw(rng):
    spread = lambda low, high: min(high, max(low, int(round(low * (high / low) ** rng.random()))))
    T, N, K = spread(1, 2600), spread(1, 2600), 8 * spread(1, 400)
    R, L = 8 * spread(1, 32), spread(1, 150)
    gated = rng.random() < 0.4
    c = _make(T, N, K, R, L, DT[rng.choice(("bf16", "f16"))], rng.choice(("none", "one", "runs", "random", "holes")), gated,
              bias=rng.random() < 0.5, residual=rng.random() < 0.5, func=rng.randrange(5), scale=rng.random() < 0.7, seed=rng.randrange(1 << 30))
    if gated and rng.random() < 0.3:
        for key in rng.choice((("a", "b"), ("a_mul", "b_mul"))):
            c[key] = None
    if rng.random() < 0.3:  # rows apart from one another
        for key in ("x", "residual"):
            if c[key] is not None:
                c[key] = torch.nn.functional.pad(c[key], (0, 8 * rng.randint(0, 3)))[:, :c[key].shape[1]]
    return c


@pytest.mark.parametrize("seed", range(12))
def test_drawn(cuda_lib, seed):
    rng = random.Random(seed)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cases = [_draw(rng) for _ in range(10)]
    outs = []
    for c in cases:
        T, N = c["x"].shape[0], c["w"].shape[0]
        wide = torch.full((T, N + rng.choice((0, 0, 1, 8))), float("nan"), dtype=c["x"].dtype, device="cuda")
        out = wide[:, :N]
        capi.moe_linear_adapters(c["x"], c["w"], out, c["ids"], a=c["a"], b=c["b"], a_mul=c["a_mul"], b_mul=c["b_mul"],
                                 scale=c["scale"], w_mul=c["w_mul"], bias=c["bias"], bias_mul=c["bias_mul"],
                                 residual=c["residual"], func=c["func"], workspace=_workspace(c), dev_status=status)
        outs.append((wide, out))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for c, (wide, out) in zip(cases, outs):
        _check(out.clone(), *_reference(c))
        assert torch.isnan(wide[:, out.shape[1]:].float()).all()


@pytest.mark.parametrize("T,N,K,R,L,gated", [(2107, 51, 2632, 48, 96, True), (1100, 40, 264, 256, 300, True), (1025, 9, 8, 8, 1000, False)])
def test_long_inputs_of_many_adapters(cuda_lib, T, N, K, R, L, gated):
    """Prompts are expected to have an adapter or two to a group of rows; many are as right."""
    c = _make(T, N, K, R, L, DT["f16"], "holes", gated, bias=True, residual=True, func=capi.MOE_FUNC_RELU, seed=T)
    out = torch.full((T, N), float("nan"), dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda o, ws: capi.moe_linear_adapters(c["x"], c["w"], o, c["ids"], a=c["a"], b=c["b"], a_mul=c["a_mul"], b_mul=c["b_mul"],
                                                  scale=c["scale"], w_mul=c["w_mul"], bias=c["bias"], bias_mul=c["bias_mul"],
                                                  residual=c["residual"], func=c["func"], workspace=ws, dev_status=status)
    call(out, _workspace(c))
    torch.cuda.synchronize()
    _check(out, *_reference(c))
    # two streams at once, a workspace each
    others, spaces, streams = [torch.empty_like(out) for _ in range(2)], [_workspace(c) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o, ws, s in zip(others, spaces, streams):
            with torch.cuda.stream(s):
                call(o, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and all(torch.equal(o, out) for o in others)
