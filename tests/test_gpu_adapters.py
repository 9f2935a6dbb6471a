"""moe_linear_adapters on the GPU against a plain 64-bit form.

Tolerances, with u = finfo.eps / 2 of the type.  Products in fp32 are off by at most one unit in the last place
(2^-23) per addition: the low-rank product v by K 2^-23 s sum |x| |a|, and 2^-22 |v| for its scale.  v enters the second
product as two numbers of the type: the first is off by u, the second holds the rest up to u of it, u^2 |v| in all (f16:
half the smallest subnormal, 2^-25, besides).  The layer's sums of K + 2 R products are off by (K + 2 R) 2^-23 of the
sum of their magnitudes.  Function, second factor, residual and the final rounding as for moe_linear: the steepest
slope of SiLU and GELU is 1.13, their fast exp adds 2^-18 |z|, and rounding is off by u.
"""
import math

import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _f(func, z):
    if func == capi.MOE_FUNC_SILU:
        return z * torch.sigmoid(z)
    if func == capi.MOE_FUNC_GELU:
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if func == capi.MOE_FUNC_GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z.clamp(min=0) if func == capi.MOE_FUNC_RELU else z


def _product(x, w, bias, a, b, scale, ids):
    """(x w^T + bias + the rows' adapters, its error bound), fp64."""
    u = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    K = x.shape[1]
    x, w = x.double(), w.double()
    z = x @ w.t() + (0 if bias is None else bias.double())
    size = x.abs() @ w.abs().t() + (0 if bias is None else bias.double().abs())
    extra = torch.zeros_like(z)
    R = 0
    if a is not None:
        R = a.shape[1]
        for j in range(a.shape[0]):
            rows = (ids == j).nonzero()[:, 0]
            if not len(rows):
                continue
            s = 1.0 if scale is None else float(scale[j])
            aj, bj = a[j].double(), b[j].double()
            v = s * (x[rows] @ aj.t())
            ev = K * 2.0 ** -23 * abs(s) * (x[rows].abs() @ aj.abs().t()) + (2.0 ** -22 + u * u) * v.abs() + tiny
            z[rows] += v @ bj.t()
            size[rows] += v.abs() @ bj.abs().t()
            extra[rows] = ev @ bj.abs().t()
    return z, (K + 2 * R) * 2.0 ** -23 * size + extra


def _reference(c):
    z, ez = _product(c["x"], c["w"], c["bias"], c["a"], c["b"], c["scale"], c["ids"])
    y = _f(c["func"], z)
    ey = 1.13 * ez + 2.0 ** -18 * z.abs()
    if c["w_mul"] is not None:
        u, eu = _product(c["x"], c["w_mul"], c["bias_mul"], c["a_mul"], c["b_mul"], c["scale"], c["ids"])
        ey = ey * u.abs() + eu * y.abs() + ey * eu
        y = y * u
    if c["residual"] is not None:
        y = y + c["residual"].double()
    return y, ey + 2.0 ** -23 * y.abs()


def _check(out, ref, bound):
    u = torch.finfo(out.dtype).eps / 2
    tiny = 2.0 ** -25 if out.dtype == torch.float16 else 0.0
    err = (out.double() - ref).abs()
    over = err - (bound + u * (ref.abs() + bound) + tiny)
    assert torch.isfinite(out.double()).all()
    assert float(over.max()) <= 0, f"off by {float(err.flatten()[over.argmax()]):.3e}"
    assert float(err.norm()) <= u * float(ref.norm()) + 1e-12


def _ids(kind, T, L, g):
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32, device="cuda")
    if kind == "one":
        return torch.full((T,), L // 2, dtype=torch.int32, device="cuda")
    if kind == "runs":
        return (torch.arange(T, device="cuda") * L // T).to(torch.int32)
    ids = torch.randint(L, (T,), generator=g, device="cuda")
    if kind == "holes":  # every third row without an adapter
        ids[torch.arange(T, device="cuda") % 3 == 1] = -1
    return ids.to(torch.int32)


def _make(T, N, K, R, L, dt, kind="random", gated=False, bias=False, residual=False, func=0, scale=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    pair = lambda: ((r(L, R, K) / math.sqrt(K)).to(dt), (r(L, N, R) * (0.5 / math.sqrt(R))).to(dt))
    a, b = pair()
    a_mul, b_mul = pair() if gated else (None, None)
    return dict(x=r(T, K).to(dt), w=(r(N, K) / math.sqrt(K)).to(dt), w_mul=(r(N, K) / math.sqrt(K)).to(dt) if gated else None,
                bias=r(N) if bias else None, bias_mul=r(N) if bias and gated else None,
                residual=r(T, N).to(dt) if residual else None, a=a, b=b, a_mul=a_mul, b_mul=b_mul,
                scale=0.5 + torch.rand(L, generator=g, device="cuda") if scale else None, ids=_ids(kind, T, L, g), func=func)


def _workspace(c):
    pairs = [t for t in (c["a"], c["a_mul"]) if t is not None]
    size = capi.moe_adapter_workspace_size(c["x"].shape[0], pairs[0].shape[1], len(pairs))
    return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type: nothing of it may be used


def _run(c, out=None, status=0, **kw):
    if out is None:
        out = torch.full((c["x"].shape[0], c["w"].shape[0]), float("nan"), dtype=c["x"].dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw.setdefault("workspace", _workspace(c))
    capi.moe_linear_adapters(c["x"], c["w"], out, c["ids"], a=c["a"], b=c["b"], a_mul=c["a_mul"], b_mul=c["b_mul"],
                             scale=c["scale"], w_mul=c["w_mul"], bias=c["bias"], bias_mul=c["bias_mul"],
                             residual=c["residual"], func=c["func"], dev_status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return out


# T, N, K, R, L: one row to many, on and off every tile, ranks below, at and above a K stage
SIZES = [(1, 1, 8, 8, 1), (1, 2048, 7168, 16, 4), (2, 64, 64, 8, 3), (3, 130, 72, 16, 2), (5, 33, 4096, 24, 5), (8, 7168, 2048, 16, 8),
         (9, 63, 1000, 40, 4), (16, 128, 512, 64, 16), (17, 129, 520, 72, 3), (31, 1000, 1544, 24, 9), (33, 96, 256, 256, 2),
         (64, 512, 1032, 128, 64), (65, 65, 520, 8, 7), (100, 2048, 256, 16, 30), (128, 256, 128, 32, 128), (129, 257, 136, 200, 2),
         (200, 4096, 512, 16, 50), (255, 1000, 2056, 48, 6), (257, 96, 64, 64, 4), (300, 7168, 264, 16, 20), (513, 1025, 520, 24, 5),
         (600, 2048, 2048, 16, 200), (1000, 200, 8, 8, 3), (1024, 2048, 1024, 64, 8), (2049, 640, 776, 80, 6), (4096, 64, 192, 16, 4),
         (5000, 1000, 512, 16, 3), (1, 70000, 64, 16, 2), (20000, 8, 64, 8, 10)]


@pytest.mark.parametrize("T,N,K,R,L", SIZES)
@pytest.mark.parametrize("form", ["plain", "gated"])
def test_sizes(cuda_lib, T, N, K, R, L, form):
    dt = DT["bf16" if (T + N) % 3 else "f16"]
    gated = form == "gated"
    kind = ("random", "runs", "holes")[(T + R // 8) % 3]
    c = _make(T, N, K, R, L, dt, kind, gated, bias=N % 2 == gated, residual=T % 2 == 1 - gated, func=(T + N + K // 8) % 5,
              seed=T + N)
    out = _run(c)
    _check(out, *_reference(c))
    assert torch.equal(out, _run(c)), "equal calls give equal bits"


@pytest.mark.parametrize("T", [1, 7, 50, 200, 1200])
@pytest.mark.parametrize("kind", ["none", "one", "runs", "random", "holes"])
@pytest.mark.parametrize("gated", [False, True])
def test_ids(cuda_lib, T, kind, gated):
    c = _make(T, 264, 328, 16, 6, DT["bf16"], kind, gated, bias=True, residual=True, func=capi.MOE_FUNC_SILU, seed=T)
    _check(_run(c), *_reference(c))


@pytest.mark.parametrize("T", [3, 90, 700])
@pytest.mark.parametrize("func", range(5))
def test_functions(cuda_lib, T, func):
    for gated in (False, True):
        c = _make(T, 200, 136, 24, 5, DT["f16"], "random", gated, residual=gated, func=func, scale=False, seed=func)
        _check(_run(c), *_reference(c))


@pytest.mark.parametrize("T", [4, 130, 900])
@pytest.mark.parametrize("which", ["w", "w_mul"])
def test_one_factor(cuda_lib, T, which):
    """Adapters of one of the two matrices only."""
    c = _make(T, 150, 256, 32, 4, DT["bf16"], "random", gated=True, func=capi.MOE_FUNC_GELU, seed=T)
    for key in ("a_mul", "b_mul") if which == "w" else ("a", "b"):
        c[key] = None
    _check(_run(c), *_reference(c))


@pytest.mark.parametrize("T", [1, 6, 100, 300, 1500])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_depend_on_their_own_adapter(cuda_lib, T, gated):
    """Infinities and NaN in an adapter (or in a row of x) stay in its rows; the others keep their bits."""
    c = _make(T, 264, 200, 16, 5, DT["bf16"], "random", gated, residual=True, seed=T)
    clean = _run(c)
    ill = 2
    for bad in ("a", "b", "scale", "a_mul", "b_mul"):
        if c[bad] is None:
            continue
        d = dict(c)
        d[bad] = c[bad].clone()
        if bad == "scale":
            d[bad][ill] = float("nan")
        else:
            d[bad][ill, 0, 3] = float("inf")
            d[bad][ill, -1, 7] = float("nan")
        out = _run(d)
        others = c["ids"] != ill
        assert torch.equal(out[others], clean[others]), bad
        if not others.all():
            rows = out[~others].double()
            assert not torch.isfinite(rows).all(1).any(), bad
            if bad == "b":  # features 0 and N - 1 alone, where the formula has them
                assert torch.isfinite(rows[:, 1:-1]).all()
    d = dict(c, x=c["x"].clone())
    d["x"][T // 2, 5] = float("nan")
    out = _run(d)
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[T // 2].double()).any()


@pytest.mark.parametrize("T", [2, 40, 800])
def test_ids_out_of_range(cuda_lib, T):
    """They set the status bit, and their rows are those of moe_linear."""
    c = _make(T, 300, 136, 16, 4, DT["bf16"], "random", seed=T)
    good = c["ids"].clone()
    c["ids"][0], c["ids"][T // 2] = 4, -2
    c["ids"][T - 1] = 2 ** 31 - 1
    out = _run(c, status=capi.MOE_DEV_BAD_ADAPTER_ID)
    bad = c["ids"] != good
    c["ids"] = torch.where(bad, -1, good).to(torch.int32)
    assert torch.equal(out, _run(c))
    _check(out, *_reference(c))


@pytest.mark.parametrize("T,N", [(1, 100), (30, 264), (260, 1000), (1030, 511)])
def test_without_adapters_is_the_layer(cuda_lib, T, N):
    """Rows without an adapter are within rounding of moe_linear's, whichever way it is launched."""
    c = _make(T, N, 520, 16, 3, DT["bf16"], "none", gated=True, bias=True, residual=True, func=capi.MOE_FUNC_SILU)
    _check(_run(c), *_reference(c))


@pytest.mark.parametrize("T", [5, 64, 400, 1100])
def test_strides_and_in_place(cuda_lib, T):
    """Rows apart from one another, adapters in slots of a larger pool, the residual replaced by the result."""
    N, K, R, L = 250, 264, 24, 5
    c = _make(T, N, K, R, L, DT["bf16"], "holes", gated=True, residual=True, func=capi.MOE_FUNC_SILU, seed=3)
    ref = _reference(c)

    def spread(t, pad, between=0):
        """A copy in a buffer with `pad` elements behind each row and `between` rows behind each matrix."""
        shape = list(t.shape)
        shape[-1] += pad
        shape[-2] += between
        big = torch.full(shape, float("nan"), dtype=t.dtype, device="cuda")
        view = big[..., :t.shape[-2], :t.shape[-1]]
        view.copy_(t)
        return view

    for key in ("x", "w", "w_mul"):
        c[key] = spread(c[key], 8)
    for key in ("a", "a_mul", "b", "b_mul"):
        c[key] = spread(c[key], 16, 3)
    wide = torch.full((T, N + 7), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 3:3 + N]
    out.copy_(c["residual"])
    c["residual"] = out
    _run(c, out=out)
    _check(out.clone(), *ref)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + N:] == 7).all()


def test_rows_behind_the_last(cuda_lib):
    """Nothing is written behind row T, nor behind the workspace."""
    for T in (1, 3, 70, 300, 1111):
        c = _make(T, 100, 72, 8, 3, DT["bf16"], seed=T)
        out = torch.full((T + 9, 100), 5.0, dtype=torch.bfloat16, device="cuda")
        size = capi.moe_adapter_workspace_size(T, 8, 1)
        ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        _run(c, out=out[:T], workspace=ws[:size])
        assert (out[T:] == 5).all() and (ws[size:] == 0x5A).all()
        _check(out[:T].clone(), *_reference(c))


@pytest.mark.parametrize("T", [4, 300])
def test_far_adapters(cuda_lib, T):
    """Offsets of adapters beyond 32 bits."""
    N, K, R = 72, 64, 8
    c = _make(T, N, K, R, 3, DT["bf16"], "random", seed=1)
    for key in ("a", "b"):
        rows, cols = c[key].shape[1:]
        step = 2 ** 31 + 8
        pool = torch.empty(2 * step + rows * cols, dtype=torch.bfloat16, device="cuda")
        far = torch.as_strided(pool, c[key].shape, (step, cols, 1))
        far.copy_(c[key])
        c[key] = far
    _check(_run(c), *_reference(c))


@pytest.mark.parametrize("T", [2, 48, 700])
def test_graph_replay_with_other_ids(cuda_lib, T):
    """Captured once, replayed with other rows and other requests."""
    c = _make(T, 136, 256, 16, 8, DT["bf16"], "random", gated=True, func=capi.MOE_FUNC_SILU, seed=1)
    ws = _workspace(c)
    out = torch.empty(T, 136, dtype=torch.bfloat16, device="cuda")
    call = lambda: capi.moe_linear_adapters(c["x"], c["w"], out, c["ids"], a=c["a"], b=c["b"], a_mul=c["a_mul"],
                                            b_mul=c["b_mul"], scale=c["scale"], w_mul=c["w_mul"], func=c["func"], workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for seed in (2, 3):
        d = _make(T, 136, 256, 16, 8, DT["bf16"], "holes" if seed == 3 else "one", seed=seed)
        c["x"].copy_(d["x"])
        c["ids"].copy_(d["ids"])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _check(out, *_reference(dict(c, bias=None, bias_mul=None, residual=None)))


def test_calls_in_a_row_and_on_streams(cuda_lib):
    """A chain of layers, each reading the last one's result, on two streams at once with a workspace each."""
    N = 256
    cs = [_make(40, N, N, 16, 6, DT["bf16"], "random", seed=s) for s in range(4)]
    first = _make(40, N, N, 16, 6, DT["bf16"], "random", seed=9)["x"]
    want = first
    for c in cs:
        want = _run(dict(c, x=want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    results = []
    for s in streams:
        ws = _workspace(cs[0])
        with torch.cuda.stream(s):
            for _ in range(5):
                x = first
                for c in cs:
                    out = torch.empty(40, N, dtype=torch.bfloat16, device="cuda")
                    capi.moe_linear_adapters(x, c["w"], out, c["ids"], a=c["a"], b=c["b"], scale=c["scale"], workspace=ws)
                    x = out
                results.append(x)
    torch.cuda.synchronize()
    assert all(torch.equal(r, want) for r in results)


def test_no_rows(cuda_lib):
    c = _make(1, 40, 64, 8, 2, DT["bf16"])
    empty = dict(c, x=c["x"][:0], ids=c["ids"][:0])
    out = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    _run(empty, out=out, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))


def test_marshalling_refuses(cuda_lib):
    c = _make(4, 40, 64, 8, 3, DT["bf16"], gated=True)
    half = lambda t: t.half()
    for kw in (dict(a=None), dict(a_mul=half(c["a_mul"])), dict(b=c["b"][:2]), dict(a=c["a"].transpose(0, 1)),
               dict(a_mul=torch.cat([c["a_mul"], c["a_mul"]], 1)[:, :8]), dict(ids=c["ids"].long()), dict(ids=c["ids"][:3]),
               dict(scale=c["scale"].double()), dict(a=c["a"].cpu())):
        with pytest.raises((ValueError, capi.MoeError)):
            _run(dict(c, **kw), workspace=_workspace(c))
    with pytest.raises(capi.MoeError) as e:
        _run(c, workspace=_workspace(c)[:-1])
    assert e.value.status == capi.MOE_ERR_WORKSPACE
