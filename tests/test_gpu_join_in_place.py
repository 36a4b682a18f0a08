"""The join's results written over what they are made from, where that is
allowed: the bits of a call with buffers of its own."""
import pytest
import torch

import test_gpu_join as join

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [(5, 136), (700, 136), (9, 2056), (400, 2056), (5, 8200), (320, 16384)]


def _same(a, b):
    assert len(a) == len(b) and all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(cuda_lib, T, H, dtype):
    c = join._case(T, 2, H, dtype, dtype, dtype)
    want = join._call(cuda_lib, c)
    x = c["x"].clone()
    _same(join._call(cuda_lib, dict(c, x=x), n=x), want)
    x = c["x"].clone()
    _same(join._call(cuda_lib, dict(c, x=x), y=x), want)
    want = cuda_lib.combine_norm(c["x"], pre=c["pre"], n_dtype=dtype)[1]
    x = c["x"].clone()
    assert torch.equal(cuda_lib.combine_norm(x, pre=c["pre"], n_dtype=dtype, n=x)[1], want)
    # a row a token, at its own place
    c = join._case(T, 1, H, dtype, dtype, dtype, pos=False, w=False)
    want = join._call(cuda_lib, c)
    for name in ("y", "n"):
        o = c["o"].clone()
        _same(join._call(cuda_lib, dict(c, o=o), **{name: o}), want)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients(cuda_lib, T, H, dtype):
    c = join._case(T, 2, H, dtype, dtype, dtype)
    want = join._call_back(cuda_lib, c)
    for name in ("dy", "dn", "x"):  # (x stands for y)
        t = c[name].clone()
        _same(join._call_back(cuda_lib, dict(c, **{name: t}), dx=t), want)


def test_overlaps_are_refused(cuda_lib):
    c = join._case(6, 2, 72, F32, F32, F32)
    buf = torch.empty(6 * 72 + 72, device="cuda")
    shifted = buf[72:].view(6, 72)
    buf[:6 * 72].view(6, 72).copy_(c["x"])
    for kw in (dict(y=shifted), dict(n=shifted)):
        with pytest.raises(cuda_lib.MoeError):
            join._call(cuda_lib, dict(c, x=buf[:6 * 72].view(6, 72)), **kw)
    with pytest.raises(cuda_lib.MoeError):
        join._call_back(cuda_lib, c, do=c["o"])
