"""moe_route_grouped where scores are smaller than fp32 holds: logits far below 0 (sigmoid, sqrt softplus), and picks far below
the largest logit (softmax with a bias), against 64 bits.

Renormalised weights are within 2e-6 of themselves: a score is off by at most 9 units of 2^-24 (exp 2, its sum 1, the
quotient 4, 2 for a root and its argument), their sum by as many and 5 for its additions, the last quotient by 4 and the
scaling by 1: 28 units, 1.7e-6.  A softmax score's argument is the rounded difference from the largest logit: half a step
of a difference d is d * 2^-24 at most, in the score and in the sum, so 2 d 2^-24 more.  Experts are those of the exact values."""
import math

import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu

SIGMOID, SQRT, SOFT_BIAS = capi.MOE_SCORE_SIGMOID, capi.MOE_SCORE_SQRTSOFTPLUS, capi.MOE_SCORE_SOFTMAX_BIAS


def _scores(logits, scoring):
    l = logits.double()
    if scoring == SOFT_BIAS:
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    return 1 / (1 + torch.exp(-l)) if scoring == SIGMOID else torch.log1p(torch.exp(l)).sqrt()


def _ref(logits, k, scoring, groups, keep, top, bias):
    s = _scores(logits, scoring)
    T, E = s.shape
    v = s if bias is None else s + bias.double()
    by = v.view(T, groups, E // groups).sort(dim=2, descending=True).values[:, :, :top].sum(2)
    kept = by.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    inside = torch.zeros_like(by, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(E // groups, 1)
    rank = logits.double() if bias is None else v  # without a bias scores order as their logits
    ids = torch.where(inside, rank, -math.inf).sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    return ids.int(), w


def _run(logits, k, scoring, renorm, groups, keep, top, bias=None, scaling=2.5, x=None, w=None):
    T, E = logits.shape
    ids, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    lo = None if x is None else torch.empty(T, E, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.moe_route_grouped(T=T, E=E, H=0 if x is None else x.shape[1], top_k=k, scoring=scoring, renormalize=renorm,
                           routed_scaling=scaling, n_group=groups, topk_group=keep, group_top=top, x=x, w_router=w,
                           logits_in=logits if x is None else None, logits_out=lo, correction_bias=bias, topk_ids=ids,
                           topk_w=wt, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return ids, wt, lo


def _check_renormalised(got, ref, difference=0, scaling=2.5):
    assert torch.equal(got[0], ref[0])
    want = ref[1] / ref[1].sum(1, keepdim=True) * scaling
    assert ((got[1].double() - want).abs() <= (2e-6 + 2 * difference * 2.0 ** -24) * want + 2.0 ** -149).all()


# one expert to a lane, up to sixteen
SHAPES = [(24, 6, 2, 2, 4), (64, 8, 3, 2, 8), (128, 1, 1, 1, 6), (180, 12, 5, 1, 6), (256, 16, 6, 2, 8), (512, 8, 3, 2, 16)]


@pytest.mark.parametrize("E,groups,keep,top,k", SHAPES)
@pytest.mark.parametrize("scoring,low,high", [(SIGMOID, -60, -30), (SIGMOID, -91, -84), (SIGMOID, -110, -88), (SIGMOID, -400, -380),
                                              (SQRT, -90, -80), (SQRT, -104, -88), (SQRT, -150, -110), (SQRT, -420, -400)])
def test_weights_of_small_scores_still_sum_up(cuda_lib, E, groups, keep, top, k, scoring, low, high):
    for T in (1, 70):
        g = torch.Generator(device="cuda").manual_seed(E + T)
        logits = torch.rand(T, E, generator=g, device="cuda") * (high - low) + low
        for bias in (None, torch.zeros(E, device="cuda"), torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1):
            got = _run(logits, k, scoring, True, groups, keep, top, bias)
            _check_renormalised(got, _ref(logits, k, scoring, groups, keep, top, bias))


@pytest.mark.parametrize("E,groups,keep,top,k", SHAPES)
@pytest.mark.parametrize("below", [30, 80, 95, 200])
def test_softmax_picks_far_below_the_largest(cuda_lib, E, groups, keep, top, k, below):
    """A bias that rules out the experts that hold the mass."""
    for T in (1, 70):
        g = torch.Generator(device="cuda").manual_seed(E + T + below)
        logits = torch.rand(T, E, generator=g, device="cuda") * 4 - below
        logits[:, ::3] += below
        bias = torch.rand(E, generator=g, device="cuda") * 0.01
        bias[::3] = -5
        got = _run(logits, k, SOFT_BIAS, True, groups, keep, top, bias)
        ref = _ref(logits, k, SOFT_BIAS, groups, keep, top, bias)
        _check_renormalised(got, ref, difference=below)


def test_small_scores_from_tokens(cuda_lib):
    for T in (1, 150):
        g = torch.Generator(device="cuda").manual_seed(T)
        x = (torch.randint(-8, 9, (T, 256), generator=g, device="cuda") / 16).bfloat16()
        w = (torch.randint(-8, 9, (128, 256), generator=g, device="cuda") / 16).bfloat16()
        x[:, 0], w[:, 0] = 16, -6  # sums of few multiples of 1 / 256: exact
        logits = x.double() @ w.double().t()
        for scoring in (SIGMOID, SQRT):
            got = _run(logits.float(), 6, scoring, True, 8, 3, 2, x=x, w=w)
            assert torch.equal(got[2].double(), logits)
            _check_renormalised(got, _ref(logits.float(), 6, scoring, 8, 3, 2, None))


@pytest.mark.parametrize("scoring,middle,spread", [(SIGMOID, -87.33, 0.05), (SIGMOID, -88.0, 1.0), (SIGMOID, -150.0, 1e-3),
                                                   (SQRT, -100.0, 0.01), (SQRT, -90.0, 1e-4), (SQRT, -103.5, 0.3),
                                                   (SQRT, -180.0, 1e-4), (SQRT, -600.0, 0.5)])
def test_groups_and_experts_of_close_small_scores(cuda_lib, scoring, middle, spread):
    """Scores that fp32 rounds to a few bits or to 0: the kept groups and the order are those of the exact values."""
    T, E, groups = 3000, 64, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = middle + (torch.rand(T, E, generator=g, device="cuda") - 0.5) * 2 * spread
    for bias in (None, torch.zeros(E, device="cuda")):
        for top in (1, 2):
            got = _run(logits, 8, scoring, True, groups, 3, top, bias)
            ref = _ref(logits, 8, scoring, groups, 3, top, bias)
            assert torch.equal(got[0], ref[0])


def test_weights_that_are_not_renormalised(cuda_lib):
    """As the scores, down to fp32's smallest normal number: 9 units of 2^-24 for the score (exp 2, its sum 1, the quotient 4,
    2 for the root and its argument), 1 for the scaling."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for scoring, low, high in ((SIGMOID, -86, -80), (SQRT, -90, -80), (SQRT, -104, -88), (SQRT, -170, -110)):
        logits = torch.rand(60, 96, generator=g, device="cuda") * (high - low) + low
        got = _run(logits, 6, scoring, False, 8, 3, 2)
        ref = _ref(logits, 6, scoring, 8, 3, 2, None)
        assert torch.equal(got[0], ref[0])
        want = ref[1] * 2.5
        assert ((got[1].double() - want).abs() <= 2e-6 * want + 2.0 ** -125).all()
