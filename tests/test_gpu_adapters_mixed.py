"""moe_linear_adapters with rows of many adapters next to prompts, at lengths where a group of rows has more items than clusters, and K
long enough for clusters: each group deals its items out in its own way."""
import pytest
import torch

from test_gpu_adapters import DT, _check, _make, _reference, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K,R,L,gated", [(1024, 40, 2080, 16, 300, False), (1025, 40, 2080, 16, 300, True), (1300, 33, 4096, 24, 90, False),
                                             (2050, 48, 2048, 64, 70, True), (300, 40, 2056, 256, 96, True), (31, 40, 2048, 256, 31, True),
                                             (5000, 24, 1544, 8, 1000, False)])
@pytest.mark.parametrize("kind", ["random", "runs", "both"])
def test_mixed_rows(cuda_lib, T, N, K, R, L, gated, kind):
    c = _make(T, N, K, R, L, DT["bf16"], "random" if kind == "random" else "runs", gated, bias=True, residual=True, func=1, seed=T)
    if kind == "both":  # one group of a prompt, one of many adapters, one of bare rows, and so on
        group = torch.arange(T, device="cuda") // 256 % 3
        ids = torch.randint(L, (T,), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
        c["ids"] = torch.where(group == 0, torch.full_like(ids, L - 1), torch.where(group == 1, ids, torch.full_like(ids, -1))).to(torch.int32)
    out = _run(c)
    _check(out, *_reference(c))
    assert torch.equal(out, _run(c)), "equal calls give equal bits"
