"""moe_linear_adapters, moe_adapter_workspace_size and moe_sandwich_norm refuse on the host, before any launch (CPU: the
pointers are never followed)."""
import ctypes

import pytest
import torch

from block_quantized_moe_router_gb300 import build, capi
from block_quantized_moe_router_gb300.layer import MoeLayer

at = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load_library()


def _adapters(lib, x=at(0x1000), w=at(0x1000), w_mul=None, bias=None, bias_mul=None, residual=None, out=at(0x8000),
              ws=at(0x9000), size=1 << 20, dims=None, status=None, **kw):
    d = capi.moe_linear_desc(4, 32, 64, 0, 0, 64, 64, 32, 32)
    for name, value in (dims or {}).items():
        setattr(d, name, value)
    ad = capi.moe_adapter_desc(3, 16, 64, 16 * 64, 16, 32 * 16, 0x2000, 0x3000, None, None, None, 0x4000)
    for name, value in kw.items():
        setattr(ad, name, value)
    return lib.moe_linear_adapters(ctypes.byref(d), ctypes.byref(ad), x, w, w_mul, bias, bias_mul, residual, out, ws, size,
                                   status, None)


def test_adapters(lib):
    assert _adapters(lib, dims=dict(T=0)) == capi.MOE_OK
    assert _adapters(lib, dims=dict(T=0), ids=None, ws=None, size=0) == capi.MOE_OK
    assert _adapters(lib, dims=dict(T=0), L=1, sa=0, sb=0) == capi.MOE_OK
    mul = dict(a_mul=0x5000, b_mul=0x6000)
    bad = [dict(L=0), dict(L=(1 << 20) + 1), dict(R=0), dict(R=12), dict(R=264, ldb=264, sb=64 * 264, sa=264 * 64), dict(lda=56), dict(lda=68),
           dict(ldb=8), dict(ldb=20), dict(sa=16 * 64 - 8), dict(sa=16 * 64 + 4), dict(sb=32 * 16 - 8), dict(sb=32 * 16 + 4),
           dict(sa=1 << 38), dict(sb=1 << 38), dict(lda=1 << 38), dict(sa=-1024), dict(a=None), dict(b=None),
           dict(a=None, b=None), dict(a_mul=0x5000), dict(b_mul=0x5000), mul, dict(mul, a=None, b=None), dict(a=0x2008),
           dict(b=0x3002), dict(w_mul=at(0x1000), a_mul=0x5008, b_mul=0x6000), dict(w_mul=at(0x1000), a_mul=0x5000, b_mul=0x6004),
           dict(ids=None), dict(ids=0x4002), dict(scale=0x4001), dict(ws=None), dict(ws=at(0x9008)), dict(out=at(0x2000)),
           dict(out=at(0x3000)), dict(out=at(0x9000)), dict(out=at(0x5000), w_mul=at(0x1000), **mul),
           dict(out=at(0x6000), w_mul=at(0x1000), **mul), dict(status=at(0x7001)),
           # and what moe_linear refuses
           dict(dims=dict(T=-1)), dict(dims=dict(K=60)), dict(dims=dict(func=5)), dict(dims=dict(dtype=2)), dict(dims=dict(ldx=56)),
           dict(x=None), dict(w=None), dict(out=None), dict(out=at(0x1000)), dict(bias_mul=at(0x7000)), dict(residual=at(0x8000), dims=dict(ldr=40))]
    for kw in bad:
        assert _adapters(lib, **kw) == capi.MOE_ERR_INVALID_ARG, kw
    need = capi.moe_adapter_workspace_size(4, 16, 1)
    assert _adapters(lib, size=need - 1) == capi.MOE_ERR_WORKSPACE
    assert _adapters(lib, w_mul=at(0x1000), size=need, **mul) == capi.MOE_ERR_WORKSPACE
    assert lib.moe_linear_adapters(None, None, None, None, None, None, None, None, None, None, 0, None, None) == capi.MOE_ERR_INVALID_ARG
    d = capi.moe_linear_desc(4, 32, 64, 0, 0, 64, 64, 32, 32)
    assert lib.moe_linear_adapters(ctypes.byref(d), None, at(0x1000), at(0x1000), None, None, None, None, at(0x8000), at(0x9000), 1 << 20,
                                   None, None) == capi.MOE_ERR_INVALID_ARG


def test_adapter_workspace(lib):
    size = capi.moe_adapter_workspace_size
    assert 0 < size(1, 8, 1) < size(100, 8, 1) < size(100, 16, 1) < size(100, 16, 2)
    assert size(1 << 30, 256, 2) >= (1 << 30) * 256 * 2 * 4
    for args in ((-1, 8, 1), ((1 << 30) + 1, 8, 1), (4, 0, 1), (4, 12, 1), (4, 264, 1), (4, 8, 0), (4, 8, 3)):
        with pytest.raises(capi.MoeError) as e:
            size(*args)
        assert e.value.status == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_adapter_workspace_size(4, 8, 1, None) == capi.MOE_ERR_INVALID_ARG


def _sandwich(lib, x=at(0x1000), r=at(0x2000), post=at(0x3000), gate=at(0x4000), row=None, w=at(0x5000), s=at(0x6000), out=at(0x7000), **kw):
    d = capi.moe_sandwich_desc(4, 32, 0, 0, 0, 1e-6, 1.0, 0.0, 32, 32, 32, 32)
    for name, value in kw.items():
        setattr(d, name, value)
    return lib.moe_sandwich_norm(ctypes.byref(d), x, r, post, gate, row, w, s, out, None)


def test_sandwich(lib):
    assert _sandwich(lib, T=0) == capi.MOE_OK
    nan, inf = float("nan"), float("inf")
    bad = [dict(T=-1), dict(H=0), dict(H=16385, ldx=20000, ldr=20000, lds=20000, ldo=20000), dict(dtype=2), dict(wide=2), dict(wide=-1),
           dict(row_sigmoid=1), dict(row_sigmoid=2, row=at(0x8000)), dict(eps=-1e-6), dict(eps=nan), dict(eps=inf), dict(residual_scale=nan),
           dict(residual_scale=inf), dict(weight_offset=nan), dict(weight_offset=-inf), dict(ldx=31), dict(ldr=31), dict(lds=31), dict(ldo=31),
           dict(ldx=1 << 38), dict(x=None), dict(s=None), dict(w=None), dict(out=None), dict(s=at(0x7000)), dict(x=at(0x1001)),
           dict(r=at(0x2001)), dict(post=at(0x3001)), dict(gate=at(0x4001)), dict(w=at(0x5001)), dict(s=at(0x6001)), dict(out=at(0x7001)),
           dict(row=at(0x8002)), dict(wide=1, r=at(0x2002)), dict(wide=1, s=at(0x6002)), dict(s=at(0x3000)), dict(s=at(0x4000)),
           dict(s=at(0x5000)), dict(out=at(0x3000)), dict(out=at(0x4000)), dict(out=at(0x5000)), dict(row=at(0x6000)), dict(row=at(0x7000)),
           dict(s=at(0x1000), lds=40), dict(s=at(0x2000), lds=40), dict(out=at(0x1000), ldo=40), dict(out=at(0x2000), ldo=40),
           dict(wide=1, s=at(0x1000)), dict(wide=1, out=at(0x2000))]
    for kw in bad:
        assert _sandwich(lib, **kw) == capi.MOE_ERR_INVALID_ARG, kw
    assert lib.moe_sandwich_norm(None, at(0x1000), None, None, None, None, None, at(0x2000), None, None) == capi.MOE_ERR_INVALID_ARG


def _layer(**kw):
    args = dict(E=24, H=256, I=128, top_k=4, scoring=capi.MOE_SCORE_SIGMOID, gate=None, up=None, down=None)
    return MoeLayer(**{**args, **kw})


class _OnGpu(torch.Tensor):
    """A tensor that says it is on a GPU."""
    @property
    def is_cuda(self):
        return True


def _mk(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnGpu)


def test_layer(lib):
    for kw in (dict(post_norm_weight=torch.ones(255, dtype=torch.bfloat16)), dict(post_norm_weight=torch.ones(256)),
               dict(block_gate=torch.ones(1, 256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            _layer(**kw)
    with pytest.raises(ValueError, match="norm_offset"):
        _layer(norm_weight=torch.ones(256, dtype=torch.bfloat16), norm_offset=1.0)
    shared = dict(gate=_mk(64, 256), up=_mk(64, 256), down=_mk(256, 64))
    good = dict(gate_a=_mk(3, 16, 256), gate_b=_mk(3, 64, 16), up_a=_mk(3, 16, 256), up_b=_mk(3, 64, 16), down_a=_mk(3, 16, 64),
                down_b=_mk(3, 256, 16), scale=_mk(3, dtype=torch.float32))
    bad = [dict(gate_a=None), dict(down_b=None), dict(gate_a=_mk(3, 12, 256), gate_b=_mk(3, 64, 12)), dict(gate_a=_mk(16, 256)),
           dict(up_a=_mk(3, 8, 256)), dict(up_b=_mk(2, 64, 16)), dict(down_a=_mk(3, 16, 256)), dict(down_b=_mk(3, 16, 256)),
           dict(gate_a=_mk(3, 16, 256, dtype=torch.float16)), dict(scale=_mk(4, dtype=torch.float32)), dict(scale=_mk(3)),
           dict(gate_a=torch.zeros(3, 16, 256, dtype=torch.bfloat16)), dict(gate_b=_mk(3, 16, 64).transpose(1, 2))]
    for kw in bad:
        with pytest.raises(ValueError, match="adapters|gate_|up_|down_"):
            _layer(shared=dict(shared, adapters={**good, **kw}))
    with pytest.raises(ValueError, match="none of"):
        _layer(shared=dict(shared, adapters=dict(scale=good["scale"])))
