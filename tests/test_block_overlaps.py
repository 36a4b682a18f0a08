"""Results that would be written over what is still to be read are refused
before anything is enqueued (no GPU needed; every call here is refused)."""
import pytest


@pytest.fixture(scope="module")
def api():
    from moe_decode_layer_gemv_gb300 import build
    build.build()
    from moe_decode_layer_gemv_gb300 import api as a
    return a


MB = 1 << 20
R, H, I, E, T, K = 8, 64, 32, 2, 4, 2


def test_the_gated_unit(api):
    def fwd(x=MB, h=2 * MB, gu=3 * MB, dt=1):
        return api._lib.moe_grouped_glu(x, 4 * MB, 5 * MB, R, H, I, E, 0, h, dt, gu, None, None)

    def back(dy=MB, gu=2 * MB, dgu=3 * MB, h=4 * MB):
        return api._lib.moe_grouped_glu_backward(dy, 5 * MB, gu, 6 * MB, R, H, I, E, 0, dgu, h, None, None)

    inv = api.MOE_ERR_INVALID_ARG
    rows, half = 2 * R * H, R * I  # bytes of x; of half of h in bf16
    for kw in (dict(h=MB), dict(h=MB + rows - 16), dict(h=MB - 2 * half + 16), dict(h=MB - 4 * half + 16, dt=0), dict(gu=MB),
               dict(gu=MB - 4 * half + 16), dict(h=3 * MB), dict(h=3 * MB + 2 * half), dict(gu=2 * MB + 16)):
        assert fwd(**kw) == inv, kw
    for kw in (dict(dgu=MB), dict(dgu=2 * MB), dict(dgu=2 * MB + 16), dict(dgu=2 * MB - 4 * half + 16), dict(h=2 * MB),
               dict(h=2 * MB + 2 * half), dict(h=MB), dict(h=MB + rows - 16), dict(h=3 * MB), dict(h=3 * MB + 4 * half - 16)):
        assert back(**kw) == inv, kw


def test_the_join(api):
    def fwd(x=MB, xd=0, o=2 * MB, od=1, pos=5 * MB, k=K, y=3 * MB, n=4 * MB, nd=1):
        return api._lib.moe_combine_norm(x, xd, o, od, pos, None, T, H, R, k, None, None, 1.0, 6 * MB, 1e-6, y, n, nd, None, None)

    def back(y=MB, yd=0, o=2 * MB, od=1, dy=3 * MB, dn=4 * MB, nd=1, dx=5 * MB, do=6 * MB):
        return api._lib.moe_combine_norm_backward(dy, dn, nd, y, yd, o, od, 7 * MB, None, T, H, R, K, None, None, 1.0, 8 * MB,
                                                  1e-6, dx, do, None, None, None, 9 * MB, 10 * MB, MB, None, None)

    inv = api.MOE_ERR_INVALID_ARG
    xn, on = 4 * T * H, 2 * R * H
    for kw in (dict(y=MB + 16), dict(y=MB - 16), dict(y=MB + xn - 16), dict(n=MB), dict(n=MB + 16), dict(n=MB + 16, nd=0),
               dict(n=3 * MB), dict(n=3 * MB + xn - 16), dict(y=MB, n=MB, nd=0), dict(y=2 * MB), dict(n=2 * MB),
               dict(n=2 * MB + on - 16), dict(y=2 * MB, xd=1), dict(y=2 * MB, pos=None, k=1), dict(n=2 * MB, nd=0, pos=None, k=1),
               dict(o=None, n=MB), dict(o=None, n=MB + 16, nd=0)):
        assert fwd(**kw) == inv, kw
    for kw in (dict(dx=3 * MB + 16), dict(dx=MB + 16), dict(dx=MB - 16), dict(dx=4 * MB), dict(dx=4 * MB + 16), dict(dx=2 * MB),
               dict(dx=2 * MB + on - 16), dict(do=2 * MB), dict(do=2 * MB + 16), dict(do=2 * MB - on + 16), dict(do=MB),
               dict(do=3 * MB), dict(do=4 * MB), dict(do=5 * MB), dict(do=5 * MB + xn - 16)):
        assert back(**kw) == inv, kw


def test_a_vector_of_scales_belongs_to_rows(api):
    import torch
    x, v = torch.zeros(4, 64), torch.zeros(64)
    for call in (lambda **kw: api.combine_norm(x, pre=v, **kw), lambda **kw: api.combine_norm_backward(x, x, x, pre=v, **kw)):
        with pytest.raises(ValueError, match="belong to rows"):
            call(scale=v)
