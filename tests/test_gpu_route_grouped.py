"""moe_route_grouped on the GPU against a plain 64-bit form: ids equal, weights within 1e-6 of the
scaling (fp32 scores: a few units in the last place; a sum of up to 512 exponentials: 2^-19.7)."""
import math

import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu

SOFTMAX, SIGMOID, SQRT, SOFT_BIAS = (capi.MOE_SCORE_SOFTMAX, capi.MOE_SCORE_SIGMOID,
                                     capi.MOE_SCORE_SQRTSOFTPLUS, capi.MOE_SCORE_SOFTMAX_BIAS)


def _ref(logits, k, scoring, renorm, scaling, groups, keep, top, bias=None):
    l = logits.double()
    fin = torch.isfinite(l)
    l = torch.where(fin, l, -math.inf)
    if scoring in (SOFTMAX, SOFT_BIAS):
        e = torch.where(fin, torch.exp(l - l.amax(1, keepdim=True)), 0.0)
        s = e / e.sum(1, keepdim=True)
    elif scoring == SIGMOID:
        s = torch.sigmoid(l)
    else:
        s = torch.nn.functional.softplus(l, threshold=50).sqrt()
    s = torch.where(fin, s, 0.0)
    v = torch.where(fin, s if bias is None or scoring == SOFTMAX else s + bias.double(), -math.inf)
    v = torch.where(torch.isfinite(v), v, -math.inf)
    T, E = v.shape
    by = v.view(T, groups, E // groups).sort(dim=2, descending=True).values[:, :, :top].sum(2)
    kept = by.sort(dim=1, descending=True, stable=True).indices[:, :keep]
    mask = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
    mask = mask.repeat_interleave(E // groups, 1)
    key = torch.where(mask, v, math.nan)
    key = torch.where(torch.isnan(key), -math.inf, torch.where(key == -math.inf, -1e300, key))
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, ids)
    if renorm:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return ids.int(), w * scaling


def _run(k, scoring, renorm, scaling, groups, keep, top, logits=None, x=None, w=None, bias=None, stream=None):
    T = logits.shape[0] if x is None else x.shape[0]
    E = logits.shape[1] if x is None else w.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    wt = torch.full((T, k), -7.0, device="cuda")
    lo = None if x is None else torch.empty(T, E, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.moe_route_grouped(T=T, E=E, H=0 if x is None else x.shape[1], top_k=k, scoring=scoring, renormalize=renorm,
                           routed_scaling=scaling, n_group=groups, topk_group=keep, group_top=top, x=x, w_router=w,
                           logits_in=logits, logits_out=lo, correction_bias=bias, topk_ids=ids, topk_w=wt,
                           dev_status=status, stream=stream)
    torch.cuda.synchronize()
    return ids, wt, lo, int(status.item())


def _agree(got, ref, scaling):
    assert torch.equal(got[0], ref[0])
    assert float((got[1].double() - ref[1]).abs().max()) <= 2e-6 * max(1.0, scaling)


# E, groups, keep, top, k
SHAPES = [(8, 1, 1, 1, 8), (8, 4, 2, 2, 3), (16, 16, 5, 1, 5), (20, 5, 2, 2, 4), (31, 1, 1, 2, 6), (60, 12, 3, 2, 7),
          (64, 64, 9, 1, 9), (96, 48, 7, 2, 14), (128, 8, 3, 2, 8), (128, 2, 1, 1, 32), (160, 5, 4, 2, 6),
          (180, 12, 5, 1, 6), (256, 16, 6, 2, 8), (256, 32, 31, 2, 10), (257, 1, 1, 1, 3), (330, 33, 4, 2, 16),
          (512, 64, 4, 2, 32), (512, 2, 1, 2, 8), (510, 3, 2, 2, 5)]


@pytest.mark.parametrize("E,groups,keep,top,k", SHAPES)
@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID, SQRT, SOFT_BIAS])
def test_from_logits(cuda_lib, E, groups, keep, top, k, scoring):
    for T in (1, 5, 33, 1000):
        g = torch.Generator(device="cuda").manual_seed(E + T)
        logits = torch.randn(T, E, generator=g, device="cuda") * 2
        for bias in (None, torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1):
            for renorm, scaling in ((True, 2.5), (False, 1.0)):
                got = _run(k, scoring, renorm, scaling, groups, keep, top, logits=logits, bias=bias)
                assert got[3] == 0
                _agree(got, _ref(logits, k, scoring, renorm, scaling, groups, keep, top, bias), scaling)


# the smallest groups that a number of experts allows with up to 64 groups
@pytest.mark.parametrize("E,groups,keep,top,k", [(33, 33, 6, 1, 6), (66, 33, 5, 2, 8), (129, 43, 5, 2, 6), (192, 64, 64, 2, 16),
                                                 (189, 63, 9, 1, 8), (260, 52, 7, 2, 9), (320, 64, 64, 2, 32),
                                                 (384, 64, 5, 1, 7), (448, 64, 9, 2, 16)])
@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID, SQRT, SOFT_BIAS])
def test_small_groups(cuda_lib, E, groups, keep, top, k, scoring):
    for T in (1, 40, 700):
        g = torch.Generator(device="cuda").manual_seed(2 * E + T)
        logits = torch.randn(T, E, generator=g, device="cuda") * 2
        for bias in (None, torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1):
            got = _run(k, scoring, True, 1.5, groups, keep, top, logits=logits, bias=bias)
            assert got[3] == 0
            _agree(got, _ref(logits, k, scoring, True, 1.5, groups, keep, top, bias), 1.5)


# E, groups, keep, top, k for many tokens, some of them odd ones
@pytest.mark.parametrize("E,groups,keep,top,k", [(128, 8, 3, 2, 8), (256, 16, 6, 2, 8), (64, 4, 1, 1, 16), (256, 32, 9, 2, 16),
                                                 (160, 8, 3, 1, 6), (8, 1, 1, 1, 8), (24, 6, 2, 2, 3), (96, 1, 1, 1, 9)])
@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID, SQRT, SOFT_BIAS])
def test_many_tokens(cuda_lib, E, groups, keep, top, k, scoring):
    T = 8200 + E % 37
    g = torch.Generator(device="cuda").manual_seed(E + k)
    logits = torch.randn(T, E, generator=g, device="cuda") * 2
    logits[5] = 0.25  # all equal
    logits[77, 3] = math.nan
    logits[78] = -math.inf
    logits[T - 1, 1] = -3.4e38
    for bias in (None, torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1, torch.zeros(E, device="cuda")):
        for renorm, scaling in ((True, 2.5), (False, 1.0)):
            got = _run(k, scoring, renorm, scaling, groups, keep, top, logits=logits, bias=bias)
            assert got[3] == capi.MOE_DEV_NONFINITE
            _agree(got, _ref(logits, k, scoring, renorm, scaling, groups, keep, top, bias), scaling)


def _grid(T, E, H, seed):
    """Tokens and a router on fixed-point grids: the logits are exact in fp32 in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = ((torch.randn(T, H, generator=g, device="cuda") * 16).round().clamp(-127, 127) / 16).bfloat16()
    w = ((torch.randn(E, H, generator=g, device="cuda") * (1.5 / math.sqrt(H)) * 4096).round().clamp(-255, 255) / 4096).bfloat16()
    return x, w


@pytest.mark.parametrize("T,E,H,groups,keep,k", [
    (1, 256, 7168, 16, 6, 8), (1, 8, 32, 2, 1, 2), (3, 180, 1184, 12, 5, 6), (8, 512, 4096, 8, 3, 8), (9, 96, 96, 8, 2, 4),
    (17, 64, 2048, 4, 2, 6), (53, 180, 1184, 12, 5, 6), (64, 256, 7168, 16, 6, 8), (127, 128, 512, 8, 4, 8),
    (128, 128, 384, 8, 4, 8), (129, 256, 1152, 4, 2, 8), (300, 384, 256, 6, 3, 8), (511, 72, 800, 3, 2, 5),
    (1000, 512, 640, 16, 4, 16), (4096, 256, 512, 16, 6, 8), (5000, 40, 32, 4, 2, 4), (9900, 96, 64, 8, 3, 5),
    (10100, 256, 128, 8, 3, 8), (2, 300, 96, 3, 2, 7), (900, 330, 160, 33, 4, 16), (7, 1, 64, 1, 1, 1),
    # blocks of experts, the last one short or ending off 16; fewer stages of K than CTAs share the tokens
    (1, 384, 7168, 8, 4, 8), (70, 272, 7584, 16, 11, 5), (161, 510, 2048, 3, 2, 9), (1500, 466, 352, 1, 1, 16),
    (5000, 257, 64, 1, 1, 4), (12000, 512, 96, 8, 3, 8), (178, 72, 160, 8, 7, 13), (245, 120, 224, 12, 5, 14),
    (128, 192, 32, 64, 9, 8), (100, 256, 64, 4, 3, 8), (640, 8, 32, 2, 1, 3)])
def test_from_tokens(cuda_lib, T, E, H, groups, keep, k):
    x, w = _grid(T, E, H, T + E)
    bias = torch.rand(E, device="cuda") * 0.2 - 0.1
    logits = x.double() @ w.double().t()
    for scoring, top in ((SIGMOID, min(2, E // groups)), (SOFTMAX, 1)):
        got = _run(k, scoring, True, 2.5, groups, keep, top, x=x, w=w, bias=bias)
        assert got[3] == 0
        assert torch.equal(got[2].double(), logits)
        _agree(got, _ref(logits, k, scoring, True, 2.5, groups, keep, top, bias), 2.5)


def test_tokens_that_are_not_finite(cuda_lib):
    """They set the status bit and disturb no other token."""
    for T in (3, 200):
        x, w = _grid(T, 128, 256, T)
        want = _run(6, SIGMOID, True, 1.0, 8, 3, 2, x=x, w=w)
        x[1, 7] = math.nan
        got = _run(6, SIGMOID, True, 1.0, 8, 3, 2, x=x, w=w)
        assert got[3] == capi.MOE_DEV_NONFINITE
        rows = [t for t in range(T) if t != 1]
        assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])
        assert got[0][1].tolist() == [0, 1, 2, 3, 4, 5] and (got[1][1] == 0).all()


def test_random_router_logits(cuda_lib):
    """Logits of ordinary values: within 1e-4 of the largest, and ids of the kernel's own logits."""
    for T in (1, 30, 700):
        x = torch.randn(T, 2048, device="cuda").bfloat16()
        w = (torch.randn(128, 2048, device="cuda") * 0.02).bfloat16()
        got = _run(6, SIGMOID, True, 1.0, 8, 3, 2, x=x, w=w)
        exact = x.double() @ w.double().t()
        assert float((got[2].double() - exact).abs().max()) <= 1e-4 * max(1.0, float(exact.abs().max()))
        _agree(got, _ref(got[2], 6, SIGMOID, True, 1.0, 8, 3, 2), 1.0)


@pytest.mark.parametrize("tokens", [4000, 9000])
@pytest.mark.parametrize("scoring", [SIGMOID, SQRT, SOFT_BIAS])
def test_scores_closer_than_fp32_can_tell(cuda_lib, scoring, tokens):
    """Pairs of experts (and of groups) whose exact values differ by less than fp32 rounding: the
    order is that of the exact values."""
    T, E, groups = tokens, 64, 8
    g = torch.Generator(device="cuda").manual_seed(11)
    bias = torch.rand(E, generator=g, device="cuda") * 0.2 - 0.1
    logits = torch.randn(T, E, generator=g, device="cuda") * 0.5
    if scoring == SOFT_BIAS:
        bias = bias * 0.1
        z = torch.exp(logits.double()).sum(1)
    a, b = torch.randint(0, E, (2, T), generator=g, device="cuda")
    rows = torch.arange(T, device="cuda")
    la = logits[rows, a].double() + 2
    for _ in range(1 if scoring != SOFT_BIAS else 4):
        if scoring == SIGMOID:
            want = (torch.sigmoid(la) + bias[a].double() - bias[b].double()).clamp(1e-3, 1 - 1e-3)
            lb = torch.log(want / (1 - want))
        elif scoring == SQRT:
            want = (torch.nn.functional.softplus(la).sqrt() + bias[a].double() - bias[b].double()).clamp(min=1e-3)
            lb = torch.log(torch.expm1(want * want))
        else:  # the pair moves the denominator: a few rounds
            logits[rows, a] = la.float()
            z = torch.exp(logits.double()).sum(1)
            lb = torch.log((torch.exp(la) / z + bias[a].double() - bias[b].double()).clamp(min=1e-4) * z)
        logits[rows, a] = la.float()
        logits[rows, b] = lb.float()
    for top in (1, 2):
        got = _run(8, scoring, True, 1.0, groups, 3, top, logits=logits, bias=bias)
        _agree(got, _ref(logits, 8, scoring, True, 1.0, groups, 3, top, bias), 1.0)


def test_offsets_beyond_32_bits(cuda_lib):
    """The last of 4.3 million tokens' logits lie 2^31 elements from the first."""
    T, E = (1 << 31) // 512 + 1000, 512
    logits = torch.zeros(T, E, device="cuda")
    rows = torch.randn(1000, E, device="cuda")
    logits[-1000:] = rows
    got = _run(3, SIGMOID, True, 1.0, 8, 2, 2, logits=logits)
    assert got[3] == 0
    assert (got[0][:-1000] == torch.tensor([0, 1, 2], device="cuda")).all()
    _agree((got[0][-1000:], got[1][-1000:]), _ref(rows, 3, SIGMOID, True, 1.0, 8, 2, 2), 1.0)


def test_ties_go_to_the_lowest(cuda_lib):
    for bias in (None, torch.zeros(64, device="cuda")):
        logits = torch.zeros(9, 64, device="cuda")
        logits[4, 40:48] = 1.0  # one group ahead, equal inside
        for scoring in (SOFTMAX, SIGMOID, SQRT, SOFT_BIAS):
            for top in (1, 2):
                got = _run(10, scoring, True, 1.0, 8, 2, top, logits=logits, bias=bias)
                first = list(range(10))
                for t in range(9):
                    assert got[0][t].tolist() == ([40, 41, 42, 43, 44, 45, 46, 47, 0, 1] if t == 4 else first)


def test_nonfinite_logits(cuda_lib):
    g = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn(7, 40, generator=g, device="cuda")
    logits[1, 3] = math.nan
    logits[2, 8:16] = math.inf      # a whole group
    logits[3, :] = -math.inf        # a whole token
    logits[4, 1:] = math.nan        # one finite logit in all
    logits[5, :] = -3.4e38          # the type's lowest value
    logits[6, ::2] = -3.4e38
    bias = torch.rand(40, generator=g, device="cuda")
    for scoring in (SOFTMAX, SIGMOID, SQRT, SOFT_BIAS):
        for b in (None, bias):
            for top in (1, 2):
                for renorm in (True, False):
                    got = _run(6, scoring, renorm, 1.5, 5, 2, top, logits=logits, bias=b)
                    assert got[3] == capi.MOE_DEV_NONFINITE
                    _agree(got, _ref(logits, 6, scoring, renorm, 1.5, 5, 2, top, b), 1.5)


def test_bias_that_is_not_finite(cuda_lib):
    logits = torch.randn(50, 32, device="cuda")
    for bad in (-math.inf, math.inf, math.nan):
        bias = torch.zeros(32, device="cuda")
        bias[::3] = bad
        got = _run(4, SIGMOID, True, 1.0, 4, 2, 2, logits=logits, bias=bias)
        assert ((got[0] % 3) != 0).all()
        _agree(got, _ref(logits, 4, SIGMOID, True, 1.0, 4, 2, 2, bias), 1.0)


def test_one_group_is_plain_routing(cuda_lib):
    logits = torch.randn(300, 96, device="cuda")
    for scoring in (SOFTMAX, SIGMOID):
        got = _run(6, scoring, True, 1.0, 1, 1, 1, logits=logits)
        ids, w = torch.empty_like(got[0]), torch.empty_like(got[1])
        capi.moe_route(T=300, E=96, H=0, top_k=6, scoring=scoring, renormalize=True, routed_scaling=1.0,
                       logits_in=logits, topk_ids=ids, topk_w=w)
        assert torch.equal(ids, got[0]) and torch.allclose(w, got[1], atol=1e-6)


def test_streams_and_graphs(cuda_lib):
    for T in (2, 40, 600):
        xs = [_grid(T, 128, 512, s) for s in range(2)]
        want = [_run(6, SIGMOID, True, 1.0, 8, 3, 2, x=x, w=w) for x, w in xs]
        s = torch.cuda.Stream()
        got = _run(6, SIGMOID, True, 1.0, 8, 3, 2, x=xs[1][0], w=xs[1][1], stream=s)
        assert torch.equal(got[0], want[1][0]) and torch.equal(got[1], want[1][1])
        x, w = xs[0][0].clone(), xs[0][1].clone()
        ids, wt, lo = (torch.empty_like(t) for t in want[0][:3])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            capi.moe_route_grouped(T=T, E=128, H=512, top_k=6, scoring=SIGMOID, renormalize=True, routed_scaling=1.0,
                                   n_group=8, topk_group=3, group_top=2, x=x, w_router=w, logits_out=lo,
                                   topk_ids=ids, topk_w=wt)
        for i in (1, 0, 1):
            x.copy_(xs[i][0])
            w.copy_(xs[i][1])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(ids, want[i][0]) and torch.equal(wt, want[i][1]) and torch.equal(lo, want[i][2])


def test_refusals(cuda_lib):
    logits = torch.zeros(2, 64, device="cuda")
    good = dict(k=4, scoring=SIGMOID, renorm=True, scaling=1.0, groups=8, keep=2, top=2, logits=logits)
    for kw in (dict(groups=0), dict(groups=7), dict(groups=65), dict(keep=0), dict(keep=9), dict(top=0), dict(top=3),
               dict(groups=64, keep=8), dict(k=17), dict(scoring=capi.MOE_SCORE_HASH), dict(scoring=9)):
        with pytest.raises(capi.MoeError):
            _run(**dict(good, **kw))
    with pytest.raises(ValueError):
        _run(**dict(good, logits=logits.half()))
    with pytest.raises(ValueError):
        _run(**dict(good, bias=torch.zeros(63, device="cuda")))
