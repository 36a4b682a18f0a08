"""The grouped products' and NVFP4 operators' refusals: made on the host
before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def api():
    from moe_decode_layer_gemv_gb300 import build
    build.build()
    from moe_decode_layer_gemv_gb300 import api as a
    return a


GOOD, ODD = 0x10000, 0x10008


@pytest.mark.parametrize("fn", ["moe_grouped_gemm", "moe_grouped_gemm_dx", "moe_grouped_gemm_dw"])
def test_grouped_products_refuse_before_any_launch(api, fn):
    f = getattr(api._lib, fn)

    def call(a=GOOD, b=GOOD, off=GOOD, R=4, N=64, K=64, E=8, out=GOOD, dt=1, st=None):
        ws = (GOOD, 0) if fn == "moe_grouped_gemm_dw" else ()
        return f(a, b, off, R, N, K, E, out, dt, *ws, st, None)

    inv = api.MOE_ERR_INVALID_ARG
    for kw in (dict(R=-1), dict(R=(1 << 22) + 1), dict(N=0), dict(N=12), dict(N=32776), dict(K=4), dict(K=20),
               dict(K=16392), dict(E=0), dict(E=257), dict(dt=2), dict(dt=-1), dict(a=None), dict(b=None),
               dict(off=None), dict(out=None), dict(a=ODD), dict(b=ODD), dict(off=ODD), dict(out=ODD), dict(st=ODD)):
        assert call(**kw) == inv, kw
    if fn != "moe_grouped_gemm_dw":  # nothing to do: no pointer is looked at
        assert call(R=0, a=None, b=None, off=None, out=None) == api.MOE_OK
    else:
        assert call(R=0, out=None) == inv


def test_split_weight_gradients_need_their_workspace(api):
    n = ctypes.c_size_t(0)
    need = api._lib.moe_grouped_gemm_dw_workspace_bytes
    assert need(1000, 64, 64, 8, ctypes.byref(n)) == 0 and n.value == 0
    assert need(1 << 16, 64, 64, 1, ctypes.byref(n)) == 0 and n.value >= 2 * 64 * 64 * 4
    assert need(1 << 16, 64, 60, 1, ctypes.byref(n)) == api.MOE_ERR_INVALID_ARG
    assert need(1 << 16, 64, 64, 1, None) == api.MOE_ERR_INVALID_ARG

    def dw(ws, nw):
        return api._lib.moe_grouped_gemm_dw(GOOD, GOOD, GOOD, 1 << 16, 64, 64, 1, GOOD, 0, ws, nw, None, None)

    assert dw(None, 1 << 30) == api.MOE_ERR_WORKSPACE and dw(GOOD, 64) == api.MOE_ERR_WORKSPACE
    assert dw(ODD, 1 << 30) == api.MOE_ERR_INVALID_ARG


def test_quantisation_refuses_before_any_launch(api):
    n = ctypes.c_size_t(0)
    ws = api._lib.moe_quantize_nvfp4_workspace_bytes
    assert ws(5, 1, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert ws(5, 7, 64, ctypes.byref(n)) == 0 and n.value >= 20
    inv = api.MOE_ERR_INVALID_ARG
    assert ws(5, 7, 64, None) == inv

    def quant(x=GOOD, dt=0, G=5, rows=7, cols=64, q=GOOD, bs=GOOD, gs=GOOD, w=GOOD, nw=1 << 20, st=None):
        return api._lib.moe_quantize_nvfp4(x, dt, G, rows, cols, q, bs, gs, w, nw, st, None)

    def dequant(q=GOOD, bs=GOOD, gs=GOOD, G=5, rows=7, cols=64, x=GOOD, dt=0):
        return api._lib.moe_dequantize_nvfp4(q, bs, gs, G, rows, cols, x, dt, None)

    for kw in (dict(G=-1), dict(G=65536), dict(rows=0), dict(rows=32769), dict(cols=16), dict(cols=48),
               dict(cols=16416), dict(dt=3), dict(x=None), dict(q=None), dict(bs=None), dict(gs=None), dict(x=ODD),
               dict(x=GOOD + 16), dict(q=ODD), dict(bs=ODD), dict(gs=ODD)):
        assert quant(**kw) == inv, kw
        assert dequant(**kw) == inv, kw
    assert quant(rows=1, G=(1 << 22) + 1) == inv
    assert quant(st=ODD) == inv and quant(w=ODD) == inv
    assert quant(w=None) == api.MOE_ERR_WORKSPACE and quant(nw=8) == api.MOE_ERR_WORKSPACE
    assert quant(G=0, x=None) == 0 and dequant(G=0, x=None) == 0


def test_nvfp4_product_refuses_before_any_launch(api):
    names = ("xq", "xbs", "xgs", "wq", "wbs", "wgs", "off")

    def call(R=4, N=64, K=64, E=8, out=GOOD, dt=0, st=None, **ptr):
        return api._lib.moe_grouped_gemm_nvfp4(*[ptr.get(n, GOOD) for n in names], R, N, K, E, out, dt, st, None)

    inv = api.MOE_ERR_INVALID_ARG
    for kw in (dict(R=-1), dict(N=12), dict(K=16), dict(K=48), dict(K=16416), dict(E=0), dict(E=257), dict(dt=2),
               dict(out=None), dict(out=ODD), dict(st=ODD), *[{n: v} for n in names for v in (None, ODD)]):
        assert call(**kw) == inv, kw
    assert call(R=0, xq=None) == api.MOE_OK


def test_the_binding_checks_tensors(api):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    off = z(9, dt=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        api.grouped_gemm(z(4, 64), z(8, 32, 64), off)
    with pytest.raises(TypeError):
        api.grouped_gemm(z(4, 64, dt=torch.float32), z(8, 32, 64), off)
    with pytest.raises(ValueError):
        api.grouped_gemm(z(4, 2, 64), z(8, 32, 64), off)
    with pytest.raises(ValueError):
        api.grouped_gemm_dx(z(4, 32), z(8, 32, 64), off)
    with pytest.raises(ValueError):
        api.grouped_gemm_dw(z(4, 32), z(4, 64), off)
    with pytest.raises(ValueError):
        api.quantize_nvfp4(z(4, 64))
    with pytest.raises(TypeError):
        api.quantize_nvfp4(z(4, 64, dt=torch.float16))
    with pytest.raises(ValueError):
        api.quantize_nvfp4(z(64))
    u8 = lambda *s: z(*s, dt=torch.uint8)  # noqa: E731
    with pytest.raises(ValueError):
        api.dequantize_nvfp4(u8(4, 32), u8(4, 4), z(4, dt=torch.float32))
    with pytest.raises(ValueError):
        api.grouped_gemm_nvfp4(u8(4, 32), u8(4, 4), z(4, dt=torch.float32), u8(8, 16, 32), u8(8, 16, 4),
                               z(8, dt=torch.float32), off)
