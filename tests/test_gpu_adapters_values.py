"""moe_linear_adapters with low-rank products that the layer's type does not hold, and with infinities in them, value by value against
the formula.  Sizes at which few rows and many go to different kernels.  Where results are finite the tolerances are those of
test_gpu_adapters; infinities, NaN and zeros are equal."""
import pytest
import torch

from test_gpu_adapters import DT, _check, _make, _reference, _run
from block_quantized_moe_router_gb300 import capi

pytestmark = pytest.mark.gpu

SIZES = [(5, 264, 200, 16), (130, 520, 264, 24), (2600, 264, 200, 16), (3000, 520, 264, 72)]
MANY = SIZES[2:]


def _product(x, w, a, b, scale, ids, L):
    """x w^T and the rows' adapters in fp64, by products that meet nothing but their own factors."""
    z = x.double() @ w.double().t()
    for j in range(L):
        rows = (ids == j).nonzero()[:, 0]
        for part in rows.split(256):
            v = (x[part].double()[:, None, :] * a[j].double()[None]).sum(-1) * float(scale[j])
            z[part] += (v[:, None, :] * b[j].double()[None]).sum(-1)
    return z


@pytest.mark.parametrize("T,N,K,R", MANY)
@pytest.mark.parametrize("form", ["plain", "first", "second"])
def test_products_beyond_f16(cuda_lib, T, N, K, R, form):
    """Two of the adapters have large scales and small b: some of a row's products exceed 65504, others do not, results are of ordinary
    size.  In the gated form the adapters of one matrix alone, so that the results stay in range."""
    c = _make(T, N, K, R, 5, DT["f16"], "holes", gated=form != "plain", residual=True, seed=T + R)
    c["scale"][1], c["scale"][3] = 1.2e5, 4e5
    for key in ("b", "b_mul"):
        if c[key] is not None:
            c[key][1:4:2] *= 1e-2
    if form != "plain":
        for key in ("a", "b") if form == "second" else ("a_mul", "b_mul"):
            c[key] = None
    ref, bound = _reference(c)
    assert float(ref.abs().max()) < 60000
    out = _run(c)
    _check(out, ref, bound)
    assert torch.equal(out, _run(c))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,K,R", SIZES)
@pytest.mark.parametrize("which", ["a", "a_mul"])
def test_an_infinite_product_stays_in_its_factor(cuda_lib, dt, T, N, K, R, which):
    """One infinite element of an adapter's a: the row's first (or second) factor is infinite throughout, by the signs of b, and the
    other one what it is.  ReLU of minus infinity times a finite number is 0, not NaN."""
    c = _make(T, N, K, R, 4, DT[dt], "random", gated=True, residual=True, func=capi.MOE_FUNC_RELU, seed=T)
    ill = int(c["ids"][0])
    c[which][ill, 2, 3] = float("inf")
    z = _product(c["x"], c["w"], c["a"], c["b"], c["scale"], c["ids"], 4)
    u = _product(c["x"], c["w_mul"], c["a_mul"], c["b_mul"], c["scale"], c["ids"], 4)
    y = torch.relu(z) * u + c["residual"].double()
    out = _run(c).double()
    rows = c["ids"] == ill
    sure = ((z.abs() > 1e-3) & (u.abs() > 1e-3))[rows]
    got, want = out[rows], y[rows]
    assert bool((torch.isinf(want) & sure).any()) and bool(((torch.isfinite(want) if which == "a" else torch.isnan(want)) & sure).any())
    assert torch.equal(torch.isnan(got)[sure], torch.isnan(want)[sure])
    same = (got == want) | torch.isnan(want)  # what is finite is 0 and the residual, exactly
    assert bool(same[sure].all())
    assert torch.isfinite(out[~rows]).all()


@pytest.mark.parametrize("T,N,K,R", SIZES[:2])
@pytest.mark.parametrize("form", ["plain", "first", "second"])
def test_products_beyond_f16_of_few_rows(cuda_lib, T, N, K, R, form):
    test_products_beyond_f16(cuda_lib, T, N, K, R, form)


@pytest.mark.parametrize("T,N,K,R", [(7, 264, 328, 16), (3, 2048, 1032, 64)])
def test_small_products_of_few_rows(cuda_lib, T, N, K, R):
    """Scales so small that f16 would hold a few bits of a product: few rows take it in fp32.  No layer beside it (zero weights), so that
    the result is the adapters' alone.  Products off by K 2^-23 of their magnitudes and 2^-22 for the scale, R of them by 2^-23 each,
    the rounding by 2^-11 or half of f16's smallest step."""
    c = _make(T, N, K, R, 3, DT["f16"], "one", seed=T)
    c["w"].zero_()
    c["scale"].fill_(2.0 ** -20)
    c["b"].mul_(2.0 ** 8)
    out = _run(c).double()
    x, a, b = c["x"].double(), c["a"][1].double(), c["b"][1].double()
    v = 2.0 ** -20 * (x @ a.t())
    ref = v @ b.t()
    ev = 2.0 ** -20 * K * 2.0 ** -23 * (x.abs() @ a.abs().t()) + 2.0 ** -22 * v.abs()
    bound = ev @ b.abs().t() + (R + 1) * 2.0 ** -23 * (v.abs() @ b.abs().t())
    assert float(((out - ref).abs() - bound - 2.0 ** -11 * ref.abs() - 2.0 ** -25).max()) <= 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,K,R", SIZES)
@pytest.mark.parametrize("form", ["plain", "first", "second"])
def test_infinite_b(cuda_lib, dt, T, N, K, R, form):
    """Infinities in an adapter's b make its rows' results infinite at their features, by the signs of the products, also where a
    product is held exactly in one number of the type; the other features stay what they are."""
    gated = form != "plain"
    c = _make(T, N, K, R, 4, DT[dt], "random", gated=gated, residual=True, seed=T + 1)
    key = "b_mul" if form == "second" else "b"
    ill = int(c["ids"][0])
    c["scale"].fill_(1.0)
    for name in ("a", "a_mul"):  # small whole numbers: products are held in one number, and none is 0
        if c[name] is not None:
            c[name].zero_()
            c[name][:, :, 0] = 1.0
    c["x"][:, 0] = (torch.arange(T, device="cuda") % 5 + 1) * torch.where(torch.arange(T, device="cuda") % 2 > 0, -1.0, 1.0)
    b = c[key]
    clean, b_clean = _run(c).double(), b.clone()
    b[ill, 5, 2], b[ill, 9, R - 1], b[ill, N - 1, 0] = float("inf"), float("-inf"), float("inf")
    b[ill, 20, 1], b[ill, 20, 3] = float("inf"), float("-inf")   # infinity minus infinity
    b[ill, 30, 1], b[ill, 30, 3] = float("inf"), float("inf")
    z = _product(c["x"], c["w"], c["a"], c["b"], c["scale"], c["ids"], 4)
    y = z
    if gated:
        y = z * _product(c["x"], c["w_mul"], c["a_mul"], c["b_mul"], c["scale"], c["ids"], 4)
    y = y + c["residual"].double()
    out = _run(c).double()
    touched = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    touched[:, [5, 9, 20, 30, N - 1]] = (c["ids"] == ill)[:, None]
    assert torch.equal(torch.isnan(out), torch.isnan(y)) and bool(torch.isnan(y[touched]).any())
    assert torch.equal(out[touched & ~torch.isnan(y)], y[touched & ~torch.isnan(y)]) and not torch.isfinite(y[touched]).any()
    assert torch.equal(out[~touched], clean[~touched])
    c[key] = b_clean
    _check(_run(c), *_reference(c))


@pytest.mark.parametrize("T,N,K,R", SIZES)
def test_infinite_product_and_b(cuda_lib, T, N, K, R):
    """An infinite product (a row of x) against finite b, infinite b and zeros in b: infinite by signs, infinite, NaN."""
    c = _make(T, N, K, R, 3, DT["bf16"], "one", residual=True, seed=T + 2)
    c["w"].zero_()
    c["a"].zero_()
    c["a"][1, 0, 0], c["a"][1, 1, 1] = 1.0, 1.0  # product 0 is x[0], product 1 is x[1], the others 0
    c["x"][:, :2] = c["x"][:, :2].abs() + 0.5
    t = T - 1
    c["a"][1, 0, 0], c["scale"][1] = 2.0 ** 100, 2.0 ** 100  # times x: beyond fp32
    c["x"][:, 0] = 0
    c["x"][t, 0] = 1.0
    c["b"][1, 0, 0], c["b"][1, 1, 0], c["b"][1, 2, 0], c["b"][1, 3, 0] = 3.0, -2.0, float("inf"), 0.0
    c["b"][1, 0:4, 1:] = 0.0
    c["b"][1, 4:, 0] = 1.0
    out = _run(c).double()
    inf = float("inf")
    assert out[t, :3].tolist() == [inf, -inf, inf] and torch.isnan(out[t, 3]) and bool((out[t, 4:] == inf).all())
    rest = out[:t]
    assert torch.isnan(rest[:, 2]).all()  # 0 x infinity
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[2] = False
    assert torch.isfinite(rest[:, keep]).all()
