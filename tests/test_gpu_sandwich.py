"""moe_sandwich_norm on the GPU against a plain 64-bit form.

Tolerances, with u = finfo.eps / 2 of a tensor's type.  A norm's factor 1 / sqrt(mean + eps) is off by H 2^-24 of the
sum of squares at most (halved by the root), 2^-22 for the root and the division; the products and the sum that
follow by 2^-24 each of what they add.  So s is off by e = c |g p| + 2^-22 (|a r| + |g p|), c = H 2^-25 + 2^-20 (the
sigmoid's fast exp included), before its rounding by u; the second norm's sum of squares then by what e adds to it.
"""
import pytest
import torch

from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _make(T, H, dt, wide=False, post=True, gate=True, row=None, nxt=True, residual=True, offset=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = lambda: (1 - offset + 0.2 * r(H)).to(dt)
    return dict(x=r(T, H).to(dt), residual=(3 * r(T, H)).to(torch.float32 if wide else dt) if residual else None,
                post_weight=w() if post else None, gate=(0.5 + 0.2 * r(H)).to(dt) if gate else None,
                row_gate=None if row is None else 2 * r(T), row_sigmoid=row == "sigmoid", weight=w() if nxt else None,
                weight_offset=offset, wide=wide)


def _reference(c, scale, eps):
    """(s, its bound, out, its bound) in fp64, without the final roundings."""
    H = c["x"].shape[1]
    c1 = H * 2.0 ** -25 + 2.0 ** -20
    p = c["x"].double()
    if c["post_weight"] is not None:
        p = p / (p.square().mean(1, keepdim=True) + eps).sqrt() * (c["post_weight"].double() + c["weight_offset"])
    if c["gate"] is not None:
        p = p * c["gate"].double()
    if c["row_gate"] is not None:
        g = c["row_gate"].double()
        p = p * (torch.sigmoid(g) if c["row_sigmoid"] else g)[:, None]
    r = 0 if c["residual"] is None else scale * c["residual"].double()
    s = p + r
    es = c1 * p.abs() + 2.0 ** -22 * (p.abs() + (0 if c["residual"] is None else r.abs()))
    if c["weight"] is None:
        return s, es, None, None
    w = c["weight"].double() + c["weight_offset"]
    q = s.square().mean(1, keepdim=True) + eps
    out = s / q.sqrt() * w
    eq = (2 * s.abs() * es + es * es).mean(1, keepdim=True) / q / 2 + c1
    return s, es, out, (es / q.sqrt() * w.abs() + eq * out.abs()) * 1.01 + 2.0 ** -22 * out.abs()


def _near(got, ref, bound):
    u = torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = (got.double() - ref).abs()
    over = err - (bound + u * (ref.abs() + bound) + tiny)
    assert torch.isfinite(got.double()).all()
    assert float(over.max()) <= 0, f"off by {float(err.flatten()[over.argmax()]):.3e}"


def _call(c, sum_out, out, scale, eps, **kw):
    capi.moe_sandwich_norm(c["x"], sum_out, residual=c["residual"], post_weight=c["post_weight"], gate=c["gate"],
                           row_gate=c["row_gate"], row_sigmoid=c["row_sigmoid"], weight=c["weight"], out=out,
                           residual_scale=scale, weight_offset=c["weight_offset"], eps=eps, **kw)


def _run(c, scale=1.0, eps=1e-6, sum_out=None, out=None):
    T, H = c["x"].shape
    ref = _reference(c, scale, eps)
    nan = lambda t: torch.full((T, H), float("nan"), dtype=t, device="cuda")
    sum_out = nan(torch.float32 if c["wide"] else c["x"].dtype) if sum_out is None else sum_out
    if c["weight"] is not None and out is None:
        out = nan(c["x"].dtype)
    _call(c, sum_out, out, scale, eps)
    torch.cuda.synchronize()
    _near(sum_out, ref[0], ref[1])
    if out is not None:
        _near(out, ref[2], ref[3])
    return sum_out, out


SIZES = [(1, 1), (1, 8), (2, 7), (3, 64), (1, 7168), (5, 2050), (31, 255), (32, 256), (33, 257), (40, 512), (64, 1000), (301, 2050),
         (100, 1024), (7, 4099), (9, 8192), (3, 8200), (2, 16384), (2, 16383), (1, 12289), (5000, 64), (70001, 16), (600, 7168), (513, 1032), (520, 4096), (700, 5000), (512, 8192), (530, 2048)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("wide", [False, True])
def test_sizes(cuda_lib, T, H, wide):
    dt = DT["f16" if H % 3 == 0 else "bf16"]
    c = _make(T, H, dt, wide, seed=H, offset=float(H % 2), row=(None, "plain", "sigmoid")[T % 3])
    a = _run(c, scale=0.5)
    b = _run(c, scale=0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,H", [(3, 1536), (50, 264), (200, 1030)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("row", [None, "plain", "sigmoid"])
@pytest.mark.parametrize("nxt", [False, True])
def test_parts(cuda_lib, T, H, post, gate, row, nxt):
    """Every part of the formula with and without the others."""
    for wide in (False, True):
        for residual in (False, True):
            _run(_make(T, H, DT["bf16"], wide, post, gate, row, nxt, residual), scale=-1.25)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("pads", [(8, 8, 8, 8), (3, 3, 3, 3), (0, 1, 2, 3), (0, 0, 8, 4)])
def test_strides(cuda_lib, pads, wide):
    """Rows of every tensor at their own distance; what lies between them is left as it was."""
    for T, H in ((5, 1000), (60, 253)):
        c = _make(T, H, DT["bf16"], wide, seed=H)

        def spread(t, pad, at=0):
            big = torch.full((T, H + pad + at), 9.0, dtype=t.dtype, device="cuda")
            view = big[:, at:at + H]
            view.copy_(t)
            return big, view

        c["x"], c["residual"] = spread(c["x"], pads[0])[1], spread(c["residual"], pads[1], 1)[1]
        s_big, s = spread(c["residual"], pads[2], 1)
        o_big, o = spread(c["x"], pads[3])
        _run(c, sum_out=s, out=o)
        assert (s_big[:, H + 1:] == 9).all() and (s_big[:, :1] == 9).all() and (o_big[:, H:] == 9).all()


def test_weights_off_their_boundary(cuda_lib):
    for H in (64, 1000, 2048):
        c = _make(40, H, DT["bf16"], seed=H)
        for i, key in enumerate(("post_weight", "gate", "weight")):
            c[key] = torch.cat([c[key][:i + 1], c[key]])[i + 1:]
        _run(c)


@pytest.mark.parametrize("T,H", [(1, 512), (6, 2056), (100, 264), (50, 101)])
def test_in_place(cuda_lib, T, H):
    """The sum over the residual and the norm over x, and the other way round."""
    c = _make(T, H, DT["bf16"], seed=T)
    want = _run(c)
    d = dict(c, x=c["x"].clone(), residual=c["residual"].clone())
    _call(d, d["residual"], d["x"], 1.0, 1e-6)
    e = dict(c, x=c["x"].clone(), residual=c["residual"].clone())
    _call(e, e["x"], e["residual"], 1.0, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(d["residual"], want[0]) and torch.equal(d["x"], want[1])
    assert torch.equal(e["x"], want[0]) and torch.equal(e["residual"], want[1])
    w = _make(T, H, DT["bf16"], wide=True, seed=T)
    want = _run(w)
    f = dict(w, x=w["x"].clone(), residual=w["residual"].clone())
    _call(f, f["residual"], f["x"], 1.0, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(f["residual"], want[0]) and torch.equal(f["x"], want[1])


def test_rows_are_apart(cuda_lib):
    """A row of zeros, one of infinities and a closed gate: the others keep their bits."""
    for H in (200, 1024, 3000):
        c = _make(40, H, DT["bf16"], row="sigmoid", seed=H)
        want = _run(c)
        d = dict(c, x=c["x"].clone(), row_gate=c["row_gate"].clone())
        d["x"][3] = 0
        d["x"][7, H // 2] = float("inf")
        d["x"][9, 0] = float("nan")
        d["row_gate"][11] = -1000.0
        s, o = torch.empty_like(want[0]), torch.empty_like(want[1])
        _call(d, s, o, 1.0, 1e-6)
        torch.cuda.synchronize()
        same = torch.ones(40, dtype=torch.bool, device="cuda")
        same[[3, 7, 9, 11]] = False
        assert torch.equal(s[same], want[0][same]) and torch.equal(o[same], want[1][same])
        assert torch.equal(s[3], c["residual"][3]) and torch.equal(s[11], c["residual"][11])
        assert torch.isnan(o[7].float()).any() and torch.isnan(o[9].float()).all()
    z = dict(c, x=torch.zeros_like(c["x"]), residual=torch.zeros_like(c["residual"]))
    s, o = torch.empty_like(c["x"]), torch.empty_like(c["x"])
    _call(z, s, o, 1.0, 1e-6)
    torch.cuda.synchronize()
    assert (s == 0).all() and (o == 0).all()


def test_wide_stream_keeps_small_steps(cuda_lib):
    """What a 16-bit residual would lose: additions of 2^-12 of its size."""
    T, H = 20, 512
    c = _make(T, H, DT["bf16"], wide=True, post=False, gate=False, nxt=False)
    c["residual"] = torch.full((T, H), 16.0, device="cuda")
    c["x"] = torch.full((T, H), 2.0 ** -8, dtype=torch.bfloat16, device="cuda")
    s, _ = _run(c)
    assert (s == 16.0 + 2.0 ** -8).all()


def test_far_rows(cuda_lib):
    """Offsets beyond 2^31 elements."""
    T, H = 3, 520
    step = 2 ** 30 + 8
    c = _make(T, H, DT["bf16"], seed=5)
    want = _run(c)
    pool = torch.empty(2 * step + H, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(pool, (T, H), (step, 1))
    far.copy_(c["x"])
    s = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    _call(dict(c, x=far), s, far, 1.0, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(s, want[0]) and torch.equal(far, want[1])


def test_graph_and_stream(cuda_lib):
    c = _make(70, 1000, DT["bf16"], row="plain")
    want = _run(c)
    s, o = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        _call(c, s, o, 1.0, 1e-6)
    for _ in range(3):
        s.fill_(0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s, want[0]) and torch.equal(o, want[1])


def test_no_rows(cuda_lib):
    c = _make(1, 64, DT["bf16"])
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    capi.moe_sandwich_norm(c["x"][:0], e, weight=c["weight"], out=e.clone())
