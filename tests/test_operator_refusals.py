"""moe_route_grouped, moe_linear and moe_add_rms_norm refuse on the host, before any launch (CPU:
the pointers are never followed)."""
import ctypes

import pytest

from block_quantized_moe_router_gb300 import build, capi

P, Q = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x8000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load_library()


def _route(lib, n_group=4, topk_group=2, group_top=2, x=P, logits_in=P, logits_out=None, ids=P, w=P, **kw):
    d = capi.moe_route_desc(4, 16, 64, 3, 1, 1, 1.0, None, None, None, 0, None, 0)
    for name, value in kw.items():
        setattr(d, name, value)
    return lib.moe_route_grouped(ctypes.byref(d), n_group, topk_group, group_top, x, logits_in, logits_out,
                                 ids, w, None, None)


def test_route_grouped(lib):
    assert _route(lib, T=0) == capi.MOE_OK
    bad = [dict(n_group=0), dict(n_group=-1), dict(n_group=3), dict(n_group=65, E=130), dict(topk_group=0),
           dict(topk_group=5), dict(group_top=0), dict(group_top=3), dict(n_group=16, topk_group=4, top_k=3),
           dict(top_k=9), dict(top_k=0), dict(E=0), dict(E=513), dict(T=-1), dict(scoring=6), dict(ids=None),
           dict(w=None), dict(routed_scaling=float("inf")), dict(logits_in=None),
           dict(logits_in=None, w_router=0x1000), dict(logits_in=None, w_router=0x1008, logits_out=P),
           dict(logits_in=None, w_router=0x1000, logits_out=P, x=ctypes.c_void_p(0x1002)),
           dict(logits_in=None, w_router=0x1000, logits_out=P, H=48)]
    for kw in bad:
        assert _route(lib, **kw) == capi.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(scoring=2, vocab=5), dict(scoring=5, vocab=5), dict(zero_experts=1)):
        assert _route(lib, **kw) == capi.MOE_ERR_UNSUPPORTED, kw
    assert lib.moe_route_grouped(None, 1, 1, 1, P, P, P, P, P, None, None) == capi.MOE_ERR_INVALID_ARG


def _linear(lib, x=P, w=P, w_mul=None, bias=None, bias_mul=None, residual=None, out=Q, **kw):
    d = capi.moe_linear_desc(4, 32, 64, 0, 0, 64, 64, 32, 32)
    for name, value in kw.items():
        setattr(d, name, value)
    return lib.moe_linear(ctypes.byref(d), x, w, w_mul, bias, bias_mul, residual, out, None, None)


def test_linear(lib):
    assert _linear(lib, T=0) == capi.MOE_OK
    odd = ctypes.c_void_p(0x1008)
    bad = [dict(T=-1), dict(T=(1 << 30) + 1), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=60), dict(K=(1 << 20) + 8), dict(dtype=2),
           dict(dtype=-1), dict(func=5), dict(func=-1), dict(ldx=56), dict(ldx=68), dict(ldw=56), dict(ldw=65),
           dict(ldo=31), dict(ldr=31, residual=P), dict(ldx=1 << 38), dict(x=None), dict(w=None), dict(out=None), dict(x=odd),
           dict(w=odd), dict(w_mul=odd), dict(out=ctypes.c_void_p(0x1001)), dict(residual=ctypes.c_void_p(0x1001)),
           dict(bias_mul=P), dict(out=P, x=P), dict(out=P, x=Q, w=P), dict(out=P, x=Q, w=Q, w_mul=P),
           dict(out=P, x=Q, w=Q, residual=P, ldr=40)]
    for kw in bad:
        assert _linear(lib, **kw) == capi.MOE_ERR_INVALID_ARG, kw
    assert lib.moe_linear(None, P, P, None, None, None, None, P, None, None) == capi.MOE_ERR_INVALID_ARG


def _norm(lib, x=P, r=None, w=P, s=None, out=ctypes.c_void_p(0x2000), **kw):
    d = capi.moe_norm_desc(4, 32, 0, 1e-6, 32, 32, 32, 32)
    for name, value in kw.items():
        setattr(d, name, value)
    return lib.moe_add_rms_norm(ctypes.byref(d), x, r, w, s, out, None)


def test_add_rms_norm(lib):
    assert _norm(lib, T=0) == capi.MOE_OK
    odd = ctypes.c_void_p(0x3001)
    bad = [dict(T=-1), dict(H=0), dict(H=16385, ldx=20000, ldo=20000), dict(dtype=2), dict(eps=-1e-6),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=31), dict(ldo=31), dict(ldr=31, r=P),
           dict(lds=31, s=P), dict(x=None), dict(w=None), dict(out=None), dict(s=ctypes.c_void_p(0x2000)),
           dict(x=odd), dict(r=odd), dict(w=odd), dict(s=odd), dict(out=odd), dict(ldo=1 << 38),
           dict(out=P, ldo=40), dict(x=Q, r=P, out=P, ldo=40), dict(s=P, lds=40), dict(x=Q, r=P, s=P, lds=40),
           dict(out=P, x=Q), dict(s=P, x=Q)]
    for kw in bad:
        assert _norm(lib, **kw) == capi.MOE_ERR_INVALID_ARG, kw
    assert lib.moe_add_rms_norm(None, P, None, P, None, P, None) == capi.MOE_ERR_INVALID_ARG
