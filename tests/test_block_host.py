"""Refusals of the operators around the grouped products: made on the host
before anything is enqueued (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def api():
    from moe_decode_layer_gemv_gb300 import build
    build.build()
    from moe_decode_layer_gemv_gb300 import api as a
    return a


GOOD, ODD = 0x10000, 0x10008


def _z(*s, dt=torch.bfloat16):
    return torch.zeros(s, dtype=dt)


def test_gated_unit_refuses_before_any_launch(api):
    def fwd(x=GOOD, w=GOOD, off=GOOD, R=4, H=64, I=64, E=8, act=0, h=GOOD, dt=1, gu=GOOD, st=None):
        return api._lib.moe_grouped_glu(x, w, off, R, H, I, E, act, h, dt, gu, st, None)

    def back(x=GOOD, w=GOOD, off=GOOD, R=4, H=64, I=64, E=8, act=0, h=GOOD, gu=GOOD, dgu=GOOD + 4096, st=None):
        return api._lib.moe_grouped_glu_backward(x, w, gu, off, R, H, I, E, act, dgu, h, st, None)

    inv = api.MOE_ERR_INVALID_ARG
    both = (dict(R=-1), dict(R=(1 << 22) + 1), dict(H=0), dict(H=12), dict(H=16392), dict(I=0), dict(I=4), dict(I=20),
            dict(I=16392), dict(I=-8), dict(E=0), dict(E=257), dict(act=2), dict(act=-1),
            *[{n: v} for n in ("x", "w", "off", "h") for v in (None, ODD)], dict(gu=ODD), dict(st=ODD))
    for kw in both:
        assert fwd(**kw) == inv, kw
        assert back(**kw) == inv, kw
    assert back(dgu=GOOD) == inv  # gu itself
    assert fwd(dt=2) == inv and back(gu=None) == inv and back(dgu=None) == inv and back(dgu=ODD) == inv
    assert fwd(R=0, x=None, h=None) == api.MOE_OK and back(R=0, x=None, dgu=None) == api.MOE_OK


def test_the_binding_checks_the_gated_unit(api):
    off = _z(9, dt=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        api.grouped_glu(_z(4, 64), _z(8, 32, 64), off)
    with pytest.raises(ValueError):
        api.grouped_glu(_z(4, 64), _z(8, 31, 64), off)
    with pytest.raises(ValueError):
        api.grouped_glu(_z(4, 64), _z(32, 64), off)
    with pytest.raises(ValueError):
        api.grouped_glu(_z(4, 64), _z(8, 32, 64), off, act="relu")
    with pytest.raises(TypeError):
        api.grouped_glu(_z(4, 64, dt=torch.float16), _z(8, 32, 64), off)
    with pytest.raises(ValueError):
        api.grouped_glu_backward(_z(4, 64), _z(8, 64, 16), _z(4, 32), off)
    with pytest.raises(ValueError):
        api.grouped_glu_backward(_z(4, 64), _z(8, 64, 16), _z(4, 32), off, act="tanh")
    with pytest.raises(ValueError):
        api.grouped_glu_backward(_z(4, 64, 1), _z(8, 64, 16), _z(4, 32), off)


def test_the_join_refuses_before_any_launch(api):
    def fwd(x=GOOD, xd=0, o=GOOD, od=1, pos=GOOD, w=GOOD, T=4, H=64, R=8, k=2, post=GOOD, scale=GOOD, pre=GOOD, eps=1e-6,
            y=GOOD, n=GOOD, nd=1, st=None):
        return api._lib.moe_combine_norm(x, xd, o, od, pos, w, T, H, R, k, post, scale, 1.0, pre, eps, y, n, nd, st, None)

    def back(x=GOOD, xd=0, o=GOOD, od=1, pos=GOOD, w=GOOD, T=4, H=64, R=8, k=2, post=GOOD, scale=GOOD, pre=GOOD, eps=1e-6,
             y=GOOD, n=GOOD, nd=1, st=None, do=GOOD + 4096, dw=GOOD, dpost=GOOD, dscale=GOOD, dpre=GOOD, dy=GOOD, ws=GOOD,
             nw=1 << 30):
        return api._lib.moe_combine_norm_backward(dy, n, nd, x, xd, o, od, pos, w, T, H, R, k, post, scale, 1.0, pre, eps, y,
                                                  do, dw, dpost, dscale, dpre, ws, nw, st, None)

    inv = api.MOE_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(T=(1 << 22) + 1), dict(H=0), dict(H=12), dict(H=16392), dict(R=-1), dict(R=(1 << 22) + 1),
               dict(k=0), dict(k=9), dict(xd=2), dict(od=-1), dict(nd=5), dict(eps=-1e-3), dict(eps=1.5),
               dict(eps=float("nan")), dict(o=None, pre=None), dict(pos=None, R=7), dict(x=None), dict(y=None), dict(n=None),
               *[{v: ODD} for v in ("x", "o", "pos", "w", "post", "scale", "pre", "y", "n", "st")]):
        assert fwd(**kw) == inv, kw
        assert back(**kw) == inv, kw
    for kw in ({v: ODD} for v in ("do", "dw", "dpost", "dscale", "dpre", "dy", "ws")):
        assert back(**kw) == inv, kw
    for kw in ({v: None} for v in ("do", "dpost", "dscale", "dpre")):
        assert back(**kw) == inv, kw
    assert back(do=GOOD) == inv  # o itself
    assert back(ws=None) == api.MOE_ERR_WORKSPACE and back(nw=64) == api.MOE_ERR_WORKSPACE
    assert fwd(T=0, x=None) == api.MOE_OK


def test_the_binding_checks_the_join(api):
    f = lambda *s: _z(*s, dt=torch.float32)  # noqa: E731
    x, o, pos, w = f(4, 64), _z(8, 64), _z(4, 2, dt=torch.int32), f(4, 2)
    for bad in (lambda: api.combine_norm(x, o, pos, w),  # host tensors
                lambda: api.combine_norm(x),
                lambda: api.combine_norm(x, pos=pos, pre=f(64)),
                lambda: api.combine_norm(f(64), o, pos, w),
                lambda: api.combine_norm(x, o, pos.flatten(), w),
                lambda: api.combine_norm_backward(x, None, x, o, pos, w, pre=f(64)),
                lambda: api.combine_norm_backward(x, x, x, o, pos, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        api.combine_norm(x.half(), o, pos, w)
    with pytest.raises(TypeError):
        api.combine_norm(x, o.half(), pos, w)


def test_orthogonalisation_refuses_before_any_launch(api):
    import ctypes
    n = ctypes.c_size_t(0)
    need = api._lib.moe_orthogonalize_workspace_bytes
    inv = api.MOE_ERR_INVALID_ARG
    assert need(3, 72, 40, ctypes.byref(n)) == 0 and n.value >= 3 * (2 * 40 * 72 + 2 * 40 * 40) * 2
    assert need(3, 72, 40, None) == inv

    def call(g=GOOD, dt=0, E=3, N=72, K=40, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, out=GOOD, ws=GOOD, nw=1 << 30, st=None):
        return api._lib.moe_orthogonalize(g, dt, E, N, K, steps, a, b, c, eps, out, ws, nw, st, None)

    for kw in (dict(E=0), dict(E=257), dict(N=0), dict(K=0), dict(N=16385), dict(K=16385), dict(dt=2), dict(steps=0),
               dict(steps=17), dict(a=17.0), dict(b=-17.0), dict(c=float("nan")), dict(eps=-1.0), dict(eps=2.0),
               dict(eps=float("nan")), *[{p: v} for p in ("g", "out") for v in (None, ODD)], dict(st=ODD), dict(ws=ODD)):
        assert call(**kw) == inv, kw
        if kw.keys() & {"E", "N", "K"}:
            assert need(kw.get("E", 3), kw.get("N", 72), kw.get("K", 40), ctypes.byref(n)) == inv
    assert call(ws=None) == api.MOE_ERR_WORKSPACE and call(nw=100) == api.MOE_ERR_WORKSPACE
    for bad in (lambda: api.orthogonalize(_z(4, 8)), lambda: api.orthogonalize(_z(4)),
                lambda: api.orthogonalize(_z(4, 8), coeffs=(1.0, 2.0))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        api.orthogonalize(_z(4, 8, dt=torch.float16))
