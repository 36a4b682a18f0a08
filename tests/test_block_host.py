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
