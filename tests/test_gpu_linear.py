"""moe_linear and moe_add_rms_norm on the GPU against plain 64-bit forms.

Tolerances.  Rounding to the output type is off by at most u = finfo.eps / 2 of the value (plus half
the smallest subnormal, f16).  The fp32 sums of K products are off by at most K * 2^-23 * A with A = sum
|x| |w| (each addition loses at most one unit in the last place, truncation included); through f the
error grows by at most 1.13 (the steepest slope of SiLU and GELU), and the fast exp of the functions
adds at most 2^-18 of |z|.  Over a whole matrix the errors of one rounding average below u, so the
2-norm of the difference is held to u times the result's.
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


def _linear_ref(x, w, func, w_mul=None, bias=None, bias_mul=None, residual=None):
    """(result, error bound without the final rounding), both fp64."""
    x, w = x.double(), w.double()
    c = x.shape[1] * 2.0 ** -23
    z = x @ w.t() + (0 if bias is None else bias.double())
    ez = c * (x.abs() @ w.abs().t() + (0 if bias is None else bias.double().abs()))
    y = _f(func, z)
    ey = 1.13 * ez + 2.0 ** -18 * z.abs()
    if w_mul is not None:
        m = w_mul.double()
        u = x @ m.t() + (0 if bias_mul is None else bias_mul.double())
        eu = c * (x.abs() @ m.abs().t() + (0 if bias_mul is None else bias_mul.double().abs()))
        ey = ey * u.abs() + eu * y.abs() + ey * eu
        y = y * u
    if residual is not None:
        y = y + residual.double()
    return y, ey + 2.0 ** -23 * y.abs()


def _check(out, ref, bound, dt):
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    err = (out.double() - ref).abs()
    over = err - (bound + u * (ref.abs() + bound) + tiny)
    assert torch.isfinite(out.double()).all()
    assert float(over.max()) <= 0, f"off by {float(err.flatten()[over.argmax()]):.3e}"
    assert float(err.norm()) <= u * float(ref.norm()) + 1e-12


def _make(T, N, K, dt, gated=False, bias=False, residual=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, w = r(T, K).to(dt), (r(N, K) / math.sqrt(K)).to(dt)
    return dict(x=x, w=w, w_mul=(r(N, K) / math.sqrt(K)).to(dt) if gated else None,
                bias=r(N) if bias else None, bias_mul=r(N) if bias and gated else None,
                residual=r(T, N).to(dt) if residual else None)


def _run(a, func, **kw):
    out = kw.pop("out", None)
    if out is None:
        out = torch.full((a["x"].shape[0], a["w"].shape[0]), float("nan"), dtype=a["x"].dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.moe_linear(a["x"], a["w"], out, w_mul=a["w_mul"], bias=a["bias"], bias_mul=a["bias_mul"],
                    residual=a["residual"], func=func, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


# T, N, K: one token to many, sizes on and off every tile (64 and 128 rows, 64 of K), long and short K
SIZES = [(1, 1, 8), (1, 2048, 7168), (2, 64, 64), (3, 130, 72), (5, 1, 4096), (8, 7168, 2048), (9, 63, 1000),
         (16, 128, 512), (17, 129, 520), (31, 1000, 1544), (64, 512, 1032), (65, 65, 65 * 8), (100, 2048, 256),
         (128, 256, 128), (129, 257, 136), (200, 4096, 512), (255, 1000, 2056), (256, 512, 512), (257, 96, 64),
         (300, 7168, 264), (511, 384, 1536), (513, 1025, 520), (1000, 200, 8), (1024, 2048, 1024),
         (2049, 640, 776), (4096, 1, 64), (4100, 300, 192), (1, 70000, 64), (3, 20001, 16), (600, 33, 8200),
         (90, 64, 16384), (70000, 8, 8), (515, 1025, 64)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("form", ["plain", "gated"])
def test_sizes(cuda_lib, T, N, K, form):
    dt = DT["bf16" if (T + N) % 3 else "f16"]
    func = (T + N + K // 8) % 5
    if form == "plain":
        a = _make(T, N, K, dt, bias=N % 2 == 0, residual=T % 2 == 1)
    else:
        a = _make(T, N, K, dt, gated=True, bias=N % 2 == 1, residual=T % 2 == 0)
    out = _run(a, func)
    ref, bound = _linear_ref(func=func, **a)
    _check(out, ref, bound, dt)
    assert torch.equal(out, _run(a, func)), "equal calls give equal bits"


@pytest.mark.parametrize("T", [1, 40, 200, 1500])
@pytest.mark.parametrize("func", range(5))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_functions(cuda_lib, T, func, dtype):
    for gated in (False, True):
        a = _make(T, 192, 256, DT[dtype], gated=gated, bias=True, residual=True, seed=T + func)
        a["x"] = a["x"] * 3  # into the functions' tails
        ref, bound = _linear_ref(func=func, **a)
        _check(_run(a, func), ref, bound, DT[dtype])


# many rows of few features; and rows at multiples of 4 bytes that are none of 16, with tiles that end in them
@pytest.mark.parametrize("T,N,K", [(700, 96, 4096), (1300, 33, 2056), (2264, 160, 5848), (20000, 40, 512), (5000, 1002, 264),
                                   (3001, 2052, 200), (2500, 1986, 520), (9000, 130, 64)])
def test_tall_and_even(cuda_lib, T, N, K):
    for gated in (False, True):
        func = (T + gated) % 5
        a = _make(T, N, K, DT["f16" if gated else "bf16"], gated=gated, bias=not gated, residual=True, seed=N)
        ref, bound = _linear_ref(func=func, **a)
        _check(_run(a, func), ref, bound, a["x"].dtype)
        wide = torch.full((T, N + 6), 7.0, dtype=a["x"].dtype, device="cuda")
        res = torch.zeros(T, N + 3, dtype=a["x"].dtype, device="cuda")  # out even, the residual's rows odd
        res[:, 1:N + 1] = a["residual"]
        out = _run({**a, "residual": res[:, 1:N + 1]}, func, out=wide[:, 2:N + 2])
        _check(out, ref, bound, a["x"].dtype)
        assert (wide[:, :2] == 7).all() and (wide[:, N + 2:] == 7).all()


# the middle range, where pairs of CTAs share the rows of x: tiles of 32 to 256 rows, one, two and four parts
# of K, odd ends of every kind
@pytest.mark.parametrize("T", [33, 64, 95, 128, 129, 161, 200, 255, 256, 257, 384])
@pytest.mark.parametrize("N,K", [(7168, 1024), (2048, 2056), (513, 1544), (320, 4096), (131, 264), (5001, 2048)])
def test_middle(cuda_lib, T, N, K):
    for gated in (False, True):
        dt = DT["f16" if (T + N) % 2 else "bf16"]
        func = (T + N // 7 + gated) % 5
        a = _make(T, N, K, dt, gated=gated, bias=T % 3 == 0, residual=(T + gated) % 2 == 0, seed=T + K)
        ref, bound = _linear_ref(func=func, **a)
        out = _run(a, func)
        _check(out, ref, bound, dt)
        assert torch.equal(out, _run(a, func)), "equal calls give equal bits"


@pytest.mark.parametrize("T,N,K", [(5000, 1003, 264), (3000, 2051, 520), (2601, 515, 72), (4097, 4159, 64)])
def test_many_odd_rows(cuda_lib, T, N, K):
    """Rows at every second multiple of 2 bytes, out and residual alike, apart, and one of them aligned."""
    for gated in (False, True):
        func = (N + gated) % 5
        a = _make(T, N, K, DT["bf16" if gated else "f16"], gated=gated, bias=True, residual=True, seed=T)
        ref, bound = _linear_ref(func=func, **a)
        want = _run(a, func)
        _check(want, ref, bound, a["x"].dtype)
        for pad_out, at_out, pad_res, at_res in ((0, 0, 1, 1), (1, 1, 0, 0), (2, 1, 3, 0), (5, 4, 2, 2)):
            wide = torch.full((T, N + pad_out), 7.0, dtype=a["x"].dtype, device="cuda")
            res = torch.full((T, N + pad_res), float("nan"), dtype=a["x"].dtype, device="cuda")
            res[:, at_res:at_res + N] = a["residual"]
            out = _run({**a, "residual": res[:, at_res:at_res + N]}, func, out=wide[:, at_out:at_out + N])
            assert torch.equal(out, want)
            assert (wide[:, :at_out] == 7).all() and (wide[:, at_out + N:] == 7).all()
        own = a["residual"].clone()
        assert torch.equal(_run({**a, "residual": own}, func, out=own), want)


@pytest.mark.parametrize("T,N,K", [(1, 300, 4096), (7, 130, 2056), (70, 257, 1000), (129, 128, 64),
                                   (300, 520, 776), (2000, 700, 520)])
def test_whole_numbers_are_exact(cuda_lib, T, N, K):
    """Sums of small whole numbers are exact in fp32, and these (below 256) in bf16 too."""
    g = torch.Generator(device="cuda").manual_seed(K)
    pick = lambda rows: torch.randint(-1, 2, (rows, K), generator=g, device="cuda")
    x, w = pick(T), pick(N)
    w[:, 240:] = 0
    w[:, ::2][:, :60] = 1
    r = torch.randint(-10, 11, (T, N), generator=g, device="cuda")
    a = dict(x=x.bfloat16(), w=w.bfloat16(), w_mul=None, bias=None, bias_mul=None, residual=r.bfloat16())
    out = _run(a, capi.MOE_FUNC_NONE)
    assert torch.equal(out.double(), x.double() @ w.double().t() + r)


@pytest.mark.parametrize("T", [1, 20, 140, 600, 3000])
def test_strides_padding_and_in_place(cuda_lib, T):
    """Rows inside wider buffers: what lies between them is neither read nor written; the residual
    may be the output itself."""
    N, K = 200, 328
    a = _make(T, N, K, torch.bfloat16, gated=True, bias=True, residual=True, seed=3)
    ref, bound = _linear_ref(func=1, **a)

    def wide(t, cols, front, fill=float("nan")):
        buf = torch.full((t.shape[0] + 2, cols), fill, dtype=t.dtype, device="cuda")
        view = buf[1:-1, front:front + t.shape[1]]
        view.copy_(t)
        return buf, view

    for name, cols, front in (("x", K + 24, 8), ("w", K + 40, 16), ("w_mul", K + 40, 24)):
        a[name] = wide(a[name], cols, front)[1]
    buf, view = wide(a["residual"], N + 37, 5)  # odd rows: no vector stores
    before = buf.clone()
    a["residual"] = view
    _run(a, 1, out=view)
    _check(view, ref, bound, torch.bfloat16)
    buf[1:-1, 5:5 + N] = 0
    before[1:-1, 5:5 + N] = 0
    assert torch.equal(buf.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("T", [2, 100, 700])
def test_nan_and_infinity_stay_in_their_rows(cuda_lib, T):
    a = _make(T, 130, 200, torch.bfloat16, seed=5)
    clean = _run(a, 0)
    a["x"][1, 7] = float("nan")
    a["w"][3, 0] = float("inf")
    out = _run(a, 0)
    rows = [t for t in range(T) if t != 1]
    cols = [n for n in range(130) if n != 3]
    assert torch.isnan(out[1]).all()
    assert not torch.isfinite(out[:, 3]).any()
    assert torch.equal(out[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("T", [1, 33, 150, 1100])
def test_streams_and_graphs(cuda_lib, T):
    """Calls on two streams at once, and one captured into a graph and replayed on new inputs."""
    a, b = _make(T, 512, 1024, torch.bfloat16, gated=True, seed=1), _make(T, 512, 1024, torch.bfloat16, gated=True, seed=2)
    want = [_run(a, 1), _run(b, 1)]
    outs = [torch.empty_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c, o in zip(streams, (a, b), outs):
            capi.moe_linear(c["x"], c["w"], o, w_mul=c["w_mul"], func=1, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graph = torch.cuda.CUDAGraph()
    x, h, y = a["x"].clone(), torch.empty_like(want[0]), torch.empty(T, 1024, dtype=torch.bfloat16, device="cuda")
    down = _make(T, 1024, 512, torch.bfloat16, seed=4)["w"]
    with torch.cuda.graph(graph):
        capi.moe_linear(x, a["w"], h, w_mul=a["w_mul"], func=1)
        capi.moe_linear(h, down, y, residual=x)
    x.copy_(b["x"])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    c = dict(a, x=b["x"])
    assert torch.equal(h, _run(c, 1))
    assert torch.equal(y, _run(dict(x=h, w=down, w_mul=None, bias=None, bias_mul=None, residual=b["x"]), 0))


@pytest.mark.parametrize("T", [3, 40, 200, 600])
def test_rows_far_apart(cuda_lib, T):
    """Element offsets beyond 32 bits, in every matrix."""
    N, K = 72, 128
    a = _make(T, N, K, torch.bfloat16, residual=True, seed=T)
    ld = (1 << 33) // T // 8 * 8  # 16 GB from the first row to the last
    buf = torch.empty(ld * T, dtype=torch.bfloat16, device="cuda")
    far = lambda cols, at: buf.as_strided((T, cols), (ld, 1), at)
    x, res, out = far(K, 0), far(N, 1024), far(N, 2048)
    x.copy_(a["x"])
    res.copy_(a["residual"])
    ref, bound = _linear_ref(func=1, **a)
    capi.moe_linear(x, a["w"], out, residual=res, func=1)
    _check(out.clone(), ref, bound, torch.bfloat16)
    odd = far(N, 4097)  # off 16 bytes
    capi.moe_linear(x, a["w"], odd, residual=res, func=1)
    assert torch.equal(odd, out)
    weight = torch.ones(N, device="cuda").bfloat16()
    s, n = far(N, 6144), far(N, 8192)
    capi.moe_add_rms_norm(out, weight, n, residual=res, sum_out=s)
    s2, n2 = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    capi.moe_add_rms_norm(out.clone(), weight, n2, residual=res.clone(), sum_out=s2)
    assert torch.equal(s, s2) and torch.equal(n, n2)


def test_no_rows(cuda_lib):
    a = _make(0, 64, 64, torch.bfloat16)
    assert _run(a, 0).shape == (0, 64)
    x = a["x"]
    capi.moe_add_rms_norm(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x))


def test_refusals(cuda_lib):
    a = _make(4, 64, 64, torch.bfloat16)
    out = torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")
    bad = [dict(x=a["x"].float()), dict(w=a["w"].half()), dict(out=out[:3]), dict(out=out.cpu()),
           dict(x=a["x"][:, :63]), dict(bias=torch.zeros(63, device="cuda")),
           dict(bias=torch.zeros(64, device="cuda", dtype=torch.bfloat16)), dict(residual=out.t()),
           dict(w_mul=torch.empty(64, 72, dtype=torch.bfloat16, device="cuda")[:, :64]),
           dict(x=a["x"].t())]
    for kw in bad:
        args = dict(x=a["x"], w=a["w"], out=out)
        args.update(kw)
        with pytest.raises((ValueError, capi.MoeError)):
            capi.moe_linear(**args)
    wide = torch.empty(4, 73, dtype=torch.bfloat16, device="cuda")
    for x in (wide[:, 1:65], wide[:, :64], torch.empty(4, 12, dtype=torch.bfloat16, device="cuda")):
        with pytest.raises((ValueError, capi.MoeError)):  # a row off 16 bytes, an odd K
            capi.moe_linear(x, a["w"][:, :x.shape[1]], out)
    with pytest.raises(capi.MoeError):  # one row for all: rows would overlap
        capi.moe_linear(a["x"][:1].expand(4, 64), a["w"], out)
    for kw in (dict(func=5), dict(func=-1), dict(bias_mul=torch.zeros(64, device="cuda"))):
        with pytest.raises(capi.MoeError):
            capi.moe_linear(a["x"], a["w"], out, **kw)
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(sum_out=out)):
        with pytest.raises(capi.MoeError):
            capi.moe_add_rms_norm(a["x"], w, out, **kw)
    with pytest.raises(ValueError):
        capi.moe_add_rms_norm(a["x"], w[:63], out)


# ---- residual add and RMS norm -------------------------------------------------------------------
def _norm_check(x, w, residual, out, sum_out, eps):
    """The fp32 sum of H squares is within H * 2^-24 of itself, the root and the products within
    2^-21: together below 2^-10 * u for H <= 16384 only as (H + 16) * 2^-25; then one rounding."""
    dt, H = x.dtype, x.shape[1]
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    s = x.double() + (0 if residual is None else residual.double())
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * w.double()
    c = (H + 16) * 2.0 ** -25
    assert ((out.double() - y).abs() <= (u + c + u * c) * y.abs() + tiny).all()
    if sum_out is not None:
        assert ((sum_out.double() - s).abs() <= (u + 2.0 ** -23) * s.abs() + tiny).all()


NORM = [(1, 1), (1, 7168), (2, 7), (3, 64), (5, 1023), (4, 1024), (301, 2050), (7, 4095), (9, 8192), (33, 7168),
        (2, 8200), (2, 16384), (3, 16383), (2, 16382), (1000, 130)]


@pytest.mark.parametrize("T,H", NORM)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("with_residual", [True, False])
def test_norm(cuda_lib, T, H, dtype, with_residual):
    g = torch.Generator(device="cuda").manual_seed(T * H)
    dt = DT[dtype]
    x = (torch.randn(T, H, generator=g, device="cuda") * 2).to(dt)
    r = (torch.randn(T, H, generator=g, device="cuda") * 5).to(dt) if with_residual else None
    w = torch.randn(H, generator=g, device="cuda").to(dt)
    for eps in (1e-6, 0.5):
        out, s = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
        capi.moe_add_rms_norm(x, w, out, residual=r, sum_out=s, eps=eps)
        _norm_check(x, w, r, out, s, eps)
        alone = torch.empty_like(x)
        capi.moe_add_rms_norm(x, w, alone, residual=r, eps=eps)
        assert torch.equal(alone, out)


@pytest.mark.parametrize("H", [64, 96, 333])
def test_norm_strides_and_in_place(cuda_lib, H):
    T = 19
    g = torch.Generator(device="cuda").manual_seed(H)
    mk = lambda cols, front: torch.randn(T + 2, cols, generator=g, device="cuda").bfloat16()[1:-1, front:front + H]
    x, r = mk(H + 8, 8), mk(H + 5, 2)
    w = torch.randn(H, generator=g, device="cuda").bfloat16()
    x0, r0 = x.clone(), r.clone()
    base = r._base.clone()
    capi.moe_add_rms_norm(x, w, x, residual=r, sum_out=r, eps=1e-5)
    torch.cuda.synchronize()
    _norm_check(x0, w, r0, x, r, 1e-5)
    now = r._base.clone()
    now[1:-1, 2:2 + H] = base[1:-1, 2:2 + H]
    assert torch.equal(now, base)


def test_norm_zero_row_and_large_values(cuda_lib):
    x = torch.zeros(3, 256, device="cuda").half()
    x[1] = 60000.0
    x[2, 5] = float("inf")
    w = torch.ones(256, device="cuda").half()
    out = torch.empty_like(x)
    capi.moe_add_rms_norm(x, w, out)
    assert (out[0] == 0).all()
    assert torch.equal(out[1], torch.ones_like(out[1]))  # the squares fit in fp32
    assert torch.isnan(out[2, 5])
