"""moe_route_grouped with biases that rule experts in or out: large ones, the type's lowest value, among tokens with logits
that are not finite.  Experts are those of the exact values."""
import math

import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu

SIGMOID, SQRT, SOFT_BIAS = capi.MOE_SCORE_SIGMOID, capi.MOE_SCORE_SQRTSOFTPLUS, capi.MOE_SCORE_SOFTMAX_BIAS
LOWEST = torch.finfo(torch.float32).min


def _ref(logits, k, scoring, groups, keep, top, bias):
    l = logits.double()
    fin = torch.isfinite(l)
    l = torch.where(fin, l, -math.inf)
    if scoring == SOFT_BIAS:
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = torch.sigmoid(l) if scoring == SIGMOID else torch.log1p(torch.exp(l)).sqrt()
    v = torch.where(fin, s + bias.double(), -math.inf)
    T, E = v.shape
    by = v.view(T, groups, E // groups).sort(dim=2, descending=True).values[:, :, :top].sum(2)
    kept = by.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    inside = torch.zeros_like(by, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(E // groups, 1)
    key = torch.where(inside, v, math.nan)  # outside below everything, -inf included
    key = torch.where(torch.isnan(key), -math.inf, torch.where(key == -math.inf, -1e300, key))
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    return ids.int(), torch.nan_to_num(w / w.sum(1, keepdim=True))


def _check(logits, k, scoring, groups, keep, top, bias, nonfinite=False):
    T, E = logits.shape
    ids, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.moe_route_grouped(T=T, E=E, H=0, top_k=k, scoring=scoring, renormalize=True, routed_scaling=1.0, n_group=groups,
                           topk_group=keep, group_top=top, logits_in=logits, correction_bias=bias, topk_ids=ids, topk_w=wt,
                           dev_status=status)
    want_ids, want_w = _ref(logits, k, scoring, groups, keep, top, bias)
    assert int(status.item()) == (capi.MOE_DEV_NONFINITE if nonfinite else 0)
    assert torch.equal(ids, want_ids)
    # fp32 scores, their sum and quotient: 28 units of 2^-24 of the weight
    assert ((wt.double() - want_w).abs() <= 2e-6 * want_w + 2.0 ** -149).all()


SHAPES = [(24, 6, 2, 4), (64, 8, 3, 8), (96, 48, 7, 9), (128, 2, 1, 8), (256, 16, 6, 8), (512, 64, 5, 16)]


@pytest.mark.parametrize("E,groups,keep,k", SHAPES)
@pytest.mark.parametrize("scoring", [SIGMOID, SQRT, SOFT_BIAS])
@pytest.mark.parametrize("out", [-1e4, -1e9, -1e30, -2e38, LOWEST])
def test_experts_ruled_out(cuda_lib, E, groups, keep, k, scoring, out):
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(300, E, generator=g, device="cuda")
    size = E // groups
    for pattern in range(4):
        bias = torch.rand(E, generator=g, device="cuda") * 0.02 - 0.01
        if pattern == 0:
            bias[::3] = out                # some of every group
        elif pattern == 1:
            bias[:size] = out              # a group
            bias[-1] = out
        elif pattern == 2:
            bias[2:] = out                 # all but two experts
        else:
            bias[:] = out
        for top in (1, 2):
            _check(logits, k, scoring, groups, keep, top, bias)


@pytest.mark.parametrize("E,groups,keep,k", SHAPES)
@pytest.mark.parametrize("scoring", [SIGMOID, SQRT, SOFT_BIAS])
def test_experts_ruled_in(cuda_lib, E, groups, keep, k, scoring):
    """Two experts of a group by biases whose sum passes the largest fp32 number, the best pair in the last group."""
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(300, E, generator=g, device="cuda")
    size = E // groups
    for base in (1e6, 1.5e38, 3e38):
        bias = torch.rand(E, generator=g, device="cuda") * 0.02 - 0.01
        for j in range(groups):
            bias[j * size] = bias[j * size + 1] = base * (1 + j / 1024)
        for top in (1, 2):
            _check(logits, k, scoring, groups, keep, top, bias)


@pytest.mark.parametrize("scoring", [SIGMOID, SQRT, SOFT_BIAS])
@pytest.mark.parametrize("out", [-1e30, LOWEST])
def test_ruled_out_experts_rank_above_logits_that_are_not_finite(cuda_lib, scoring, out):
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn(40, 64, generator=g, device="cuda")
    logits[:, :16] = -math.inf             # two groups without a finite logit
    logits[::2, 3] = math.nan
    bias = torch.rand(64, generator=g, device="cuda") * 0.02
    bias[24:] = out                        # and only one that is not ruled out
    for keep, k in ((1, 8), (3, 20), (7, 32)):
        for top in (1, 2):
            _check(logits, k, scoring, 8, keep, top, bias, nonfinite=True)


def test_softmax_bias_between_close_scores(cuda_lib):
    """Pairs of experts whose biases make up for what their probabilities differ by, to within fp32's rounding, beside an
    expert that a bias rules out: the order is that of the exact values."""
    T, E = 4000, 512
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(1, E, generator=g, device="cuda") * 0.3
    p = torch.softmax(logits.double(), 1)[0]
    bias = (p.amax() - p).float()  # every sum within half a step of the same value
    bias[7] = -1e9
    _check(logits.expand(T, E).contiguous(), 16, SOFT_BIAS, 8, 3, 2, bias)
    wobble = logits + torch.randn(T, E, generator=g, device="cuda") * 1e-6
    _check(wobble, 16, SOFT_BIAS, 8, 3, 2, bias)
    _check(wobble, 8, SOFT_BIAS, 1, 1, 1, bias)


def test_a_ruled_out_expert_costs_no_more(cuda_lib):
    """One bias of -1e9 among 128: of the order of the time without it (1.07 of it measured; 27 where every token went to fp64)."""
    logits = torch.randn(32768, 128, device="cuda")
    ids, wt = torch.empty(32768, 8, dtype=torch.int32, device="cuda"), torch.empty(32768, 8, device="cuda")
    bias = torch.rand(128, device="cuda") * 0.01
    masked = bias.clone()
    masked[5] = -1e9

    def us(b):
        best = math.inf
        for _ in range(20):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            for _ in range(10):
                capi.moe_route_grouped(T=32768, E=128, H=0, top_k=8, scoring=SOFT_BIAS, renormalize=True, routed_scaling=1.0,
                                       n_group=8, topk_group=3, group_top=2, logits_in=logits, correction_bias=b,
                                       topk_ids=ids, topk_w=wt)
            end.record()
            torch.cuda.synchronize()
            best = min(best, begin.elapsed_time(end) * 100)
        return best

    plain = us(bias)
    assert us(masked) <= 4 * plain
