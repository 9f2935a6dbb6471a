"""MoeLayer.ffn with adapters on its shared expert against the formula, for the lengths that forward runs in one launch too."""
import pytest
import torch

from test_gpu_layer_adapters import _ids, _layer, _low, _shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 5, 8, 9])
@pytest.mark.parametrize("groups", [False, True])
def test_ffn(cuda_lib, T, groups):
    """On top of the routed experts alone, for the same ids and weights.  h is rounded once (2^-8 of each of its products), the routed sum
    before it (2^-8 of itself), the result once more."""
    s = _shared()
    layer, x = _layer(T, groups=groups, shared=s)
    plain, _ = _layer(T, groups=groups)
    ids = _ids(T)
    chosen, w, _ = layer.route(x)
    out = layer.ffn(x, chosen, w, adapter_ids=ids)
    routed = plain.ffn(x, chosen, w)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0
    ad = s["adapters"]
    low = lambda v, key: _low(v, ad[key + "_a"], ad[key + "_b"], ad["scale"], ids)
    z = x.double() @ s["gate"].double().t() + s["gate_bias"].double() + low(x, "gate")
    h = z * torch.sigmoid(z) * (x.double() @ s["up"].double().t() + low(x, "up"))
    want = h @ s["down"].double().t() + low(h, "down") + routed.double()
    size = h.abs() @ s["down"].double().abs().t() + routed.double().abs()
    for j in range(ad["scale"].numel()):
        rows = ids == j
        size[rows] += float(ad["scale"][j]) * (h[rows].abs() @ ad["down_a"][j].double().abs().t()) @ ad["down_b"][j].double().abs().t()
    assert float(((out.double() - want).abs() - 2.0 ** -8 * size - 2.0 ** -8 * want.abs() - 1e-4).max()) <= 0
    # forward routes by itself, in one launch for a few tokens: the same routed experts to their rounding
    there = layer.forward(x, adapter_ids=ids)[0]
    alone = plain.forward(x)[0]
    gap = (alone.double() - routed.double()).abs()
    assert float(((there.double() - out.double()).abs() - gap - 2.0 ** -7 * want.abs() - 1e-4).max()) <= 0
    for la in (layer, plain):
        la.close()
