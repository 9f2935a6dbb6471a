"""Clustered kernels with little shared memory each, on many streams at once: their CTAs share SMs and tensor memory."""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu


def test_small_products_side_by_side(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(7)
    mk = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    jobs = []
    for T, E, H in ((1, 256, 1024), (1, 129, 64), (9, 256, 128), (2048, 272, 64), (4096, 272, 64), (300, 130, 32), (64, 40, 96)):
        x, w = mk(T, H), mk(E, H)

        def route(outs, x=x, w=w, T=T, E=E, H=H):
            capi.moe_route_grouped(T=T, E=E, H=H, top_k=4, scoring=0, renormalize=True, routed_scaling=1.0, n_group=1,
                                   topk_group=1, group_top=1, x=x, w_router=w, logits_out=outs[0], topk_ids=outs[1],
                                   topk_w=outs[2], dev_status=status, stream=torch.cuda.current_stream())
        jobs.append((route, lambda T=T, E=E: (torch.empty(T, E, device="cuda"), torch.empty(T, 4, dtype=torch.int32, device="cuda"),
                                              torch.empty(T, 4, device="cuda"))))
    for T, N, K in ((1, 512, 64), (48, 1024, 64), (100, 640, 64), (128, 4096, 128), (200, 1024, 128)):
        x, w = mk(T, K), mk(N, K)
        jobs.append((lambda outs, x=x, w=w: capi.moe_linear(x, w, outs[0], dev_status=status, stream=torch.cuda.current_stream()),
                     lambda T=T, N=N: (torch.empty(T, N, dtype=torch.bfloat16, device="cuda"),)))
    want = []
    for call, room in jobs:
        want.append(room())
        call(want[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[room() for _ in range(40)] for _, room in jobs]
    torch.cuda.synchronize()
    for i in range(40):
        for (call, _), s, outs in zip(jobs, streams, got):
            with torch.cuda.stream(s):
                call(outs[i])
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for outs, ref in zip(got, want):
        for one in outs:
            assert all(torch.equal(a, b) for a, b in zip(one, ref))
