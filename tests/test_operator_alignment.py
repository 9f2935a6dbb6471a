"""moe_route_grouped and moe_linear refuse float and int32 pointers off 4 bytes on the host (CPU: the pointers are never
followed)."""
import ctypes

import pytest

from block_quantized_moe_router_gb300 import build, capi

P, Q, OUT = (ctypes.c_void_p(a) for a in (0x1000, 0x8000, 0x20000))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load_library()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_route_grouped(lib, off):
    def call(bias=None, x=None, w_router=None, logits_in=P, logits_out=None, ids=P, w=P, status=None):
        d = capi.moe_route_desc(4, 16, 64, 3, 1, 1, 1.0, w_router, bias, None, 0, None, 0)
        return lib.moe_route_grouped(ctypes.byref(d), 4, 2, 2, x, logits_in, logits_out, ids, w, status, None)

    bad = ctypes.c_void_p(0x4000 + off)
    for kw in (dict(bias=0x4000 + off), dict(logits_in=bad), dict(ids=bad), dict(w=bad), dict(status=bad),
               dict(logits_in=None, x=P, w_router=0x1000, logits_out=bad)):
        assert call(**kw) == capi.MOE_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("off", [1, 2, 3])
def test_linear(lib, off):
    bad = ctypes.c_void_p(0x4000 + off)
    d = capi.moe_linear_desc(4, 32, 64, 0, 0, 64, 64, 32, 32)
    for bias, w_mul, bias_mul, status in ((bad, None, None, None), (None, P, bad, None), (P, P, bad, None), (None, None, None, bad)):
        assert lib.moe_linear(ctypes.byref(d), P, Q, w_mul, bias, bias_mul, None, OUT, status, None) == capi.MOE_ERR_INVALID_ARG
