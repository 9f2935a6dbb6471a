"""The first launch of each new kernel in a process of its own: code, descriptors and translations are cold
then, and waits that never last in a warm process do."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, torch
from block_quantized_moe_router_gb300 import capi
what, T, N, K = sys.argv[1], int(sys.argv[2]), int(sys.argv[3]), int(sys.argv[4])
g = torch.Generator(device="cuda").manual_seed(1)
mk = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").bfloat16()
status = torch.zeros(1, dtype=torch.int32, device="cuda")
x, w = mk(T, K), mk(N, K) / 64
if what == "route":
    ids = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    tw, logits = torch.empty(T, 4, device="cuda"), torch.empty(T, N, device="cuda")
    for _ in range(3):
        capi.moe_route_grouped(T=T, E=N, H=K, top_k=4, scoring=0, renormalize=True, routed_scaling=1.0, n_group=4,
                               topk_group=2, group_top=1, x=x, w_router=w, logits_out=logits, topk_ids=ids,
                               topk_w=tw, dev_status=status)
    torch.cuda.synchronize()
    assert torch.equal(logits.double(), x.double() @ w.double().t())  # sums of few multiples of 1 / 64: exact
    assert (tw.sum(1) - 1).abs().max() < 1e-5
else:
    v = mk(N, K) / 64 if what == "gated" else None
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        capi.moe_linear(x, w, out, w_mul=v, dev_status=status)
    torch.cuda.synchronize()
    ref = x.double() @ w.double().t()
    if v is not None:
        ref = ref * (x.double() @ v.double().t())
    # the sums are exact, their product is off by 2^-24 of itself and its rounding by 2^-8
    assert ((out.double() - ref).abs() <= 1.001 * 2.0 ** -8 * ref.abs()).all()
assert status.item() == 0
print("right")
"""


@pytest.mark.parametrize("what,T,N,K", [("gated", 1, 2048, 7168), ("gated", 300, 1024, 7168), ("plain", 5, 7168, 2048),
                                        ("plain", 128, 7168, 2048), ("gated", 100, 2048, 7168),
                                        ("plain", 1000, 2048, 2048), ("route", 1, 256, 7168), ("route", 500, 64, 2048)])
def test_first_launch(cuda_lib, what, T, N, K):
    done = subprocess.run([sys.executable, "-c", CHILD, what, str(T), str(N), str(K)], cwd=ROOT, capture_output=True,
                          text=True, timeout=300, env={**os.environ, "PYTHONPATH": ROOT})
    assert done.returncode == 0 and "right" in done.stdout, done.stdout[-500:] + done.stderr[-2000:]
