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

    def back(x=GOOD, w=GOOD, off=GOOD, R=4, H=64, I=64, E=8, act=0, h=GOOD, gu=GOOD, dgu=GOOD, st=None):
        return api._lib.moe_grouped_glu_backward(x, w, gu, off, R, H, I, E, act, dgu, h, st, None)

    inv = api.MOE_ERR_INVALID_ARG
    both = (dict(R=-1), dict(R=(1 << 22) + 1), dict(H=0), dict(H=12), dict(H=16392), dict(I=0), dict(I=4), dict(I=20),
            dict(I=16392), dict(I=-8), dict(E=0), dict(E=257), dict(act=2), dict(act=-1),
            *[{n: v} for n in ("x", "w", "off", "h") for v in (None, ODD)], dict(gu=ODD), dict(st=ODD))
    for kw in both:
        assert fwd(**kw) == inv, kw
        assert back(**kw) == inv, kw
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
             y=GOOD, n=GOOD, nd=1, st=None, do=GOOD, dw=GOOD, dpost=GOOD, dscale=GOOD, dpre=GOOD, dy=GOOD, ws=GOOD,
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
