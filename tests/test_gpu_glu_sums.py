"""Long sums of one sign in the gated unit and its gradient, and what bad
offsets leave alone.

The tensor cores' truncating additions make such a sum smaller: 64 of them,
what an accumulator of the plain products takes, by 1.0e-6 (2^-20), fewer by
less in proportion.  h = g u of two sums in fp32 takes 24 an accumulator: two
times 24 / 64 of that at most, below 2^-20, no more than a plain product loses.
dh is one accumulator of H / 16 additions, 7.4e-5 for 16384 terms and for fewer
less in proportion.  Means of relative errors are compared, a bias and no
scatter; a rounding to bf16 adds 2^-8 / sqrt(3 n) at most to the mean of n
evenly spread ones, of which five are allowed (test_gpu_grouped_sums.py)."""
import pytest
import torch

import test_gpu_glu as glu

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
ROUNDINGS = 5 * 2.0 ** -8 / 3 ** 0.5


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV) + 0.5


def _spread(n):
    return 2.0 ** torch.linspace(0, 1, n, device=DEV)


CASES = [([512], 768, 16384), ([60], 768, 16384), ([300, 0, 500], 1032, 2056)]


@pytest.mark.parametrize("act", glu.ACTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("counts,I,H", CASES)
def test_gated_units_of_long_sums(cuda_lib, counts, I, H, dtype, act):
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    R, E = sum(counts), len(counts)
    x = (_rand(g, R, H) * _spread(R).unsqueeze(1)).to(BF16)
    w = (_rand(g, E, 2 * I, H) * torch.cat([_spread(I), _spread(I).flip(0)]).view(1, -1, 1)).to(BF16)
    off = torch.tensor([0, *counts], device=DEV).cumsum(0).to(torch.int32)
    h, gu = cuda_lib.grouped_glu(x, w, off, act=act, keep=True, out_dtype=dtype)
    want = torch.cat([x[a:b].double() @ w[e].double().T for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    assert float(want.min()) > 100  # act(g) = g, exactly
    bias = float((h.double() / (want[:, :I] * want[:, I:]) - 1).mean())
    # (a bf16 h is made of sums in parts of 1024 terms)
    assert abs(bias) <= (2.0 ** -20 if dtype == F32 else 2 * 2.0 ** -20 + ROUNDINGS / h.numel() ** 0.5), bias
    bias = float((gu.double() / want - 1).mean())
    assert abs(bias) <= 2.0 ** -20 + ROUNDINGS / gu.numel() ** 0.5, bias


@pytest.mark.parametrize("act", glu.ACTS)
@pytest.mark.parametrize("counts,I,H", CASES)
def test_gradients_of_long_sums(cuda_lib, counts, I, H, act):
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    R, E = sum(counts), len(counts)
    dy = (_rand(g, R, H) * _spread(R).unsqueeze(1)).to(BF16)
    down = (_rand(g, E, H, I) * _spread(I)).to(BF16)
    gu = torch.cat([100 * _rand(g, R, I), _rand(g, R, I)], 1).to(BF16)  # act(g) = g, act'(g) = 1
    off = torch.tensor([0, *counts], device=DEV).cumsum(0).to(torch.int32)
    dgu, _ = cuda_lib.grouped_glu_backward(dy, down, gu, off, act=act)
    dh = torch.cat([dy[a:b].double() @ down[e].double() for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    for got, f in ((dgu[:, :I], gu[:, I:]), (dgu[:, I:], gu[:, :I])):
        bias = float((got.double() / (dh * f.double()) - 1).mean())
        assert abs(bias) <= 7.4e-5 * H / 16384 + ROUNDINGS / dh.numel() ** 0.5, bias


@pytest.mark.parametrize("rows", [6, 60, 600])
@pytest.mark.parametrize("offsets", [[0, 4, 2, 6], [-1, 2, 3, 6], [0, 2, 3, 7], [0, 2 ** 31 - 1, 2, 6], [1, 3, 2, 2]])
def test_bad_offsets_leave_the_other_segments_right(cuda_lib, offsets, rows):
    """Rows of a good segment are right and rows of none left as they were.
    (Where good segments overlap beside a bad one, their rows are not valid.)"""
    scale = rows // 6
    offsets = [o if abs(o) > 9 else o * scale for o in offsets]
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    c = glu._case([rows, 0, 0], 40, 72)
    new = lambda w, t=BF16: torch.full((rows, w), -7.0, dtype=t, device=DEV)  # noqa: E731
    segs = [(a, b) if 0 <= a <= b <= rows else (0, 0) for a, b in zip(offsets, offsets[1:])]
    none = torch.ones(rows, dtype=torch.bool, device=DEV)
    for a, b in segs:
        none[a:b] = False
    for dtype in (F32, BF16):
        h, gu, dgu, hb = new(40, dtype), new(80), new(80), new(40)
        cuda_lib.grouped_glu(c["x"], c["w"], off, out=h, gu=gu)
        cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], off, dgu=dgu, h=hb)
        for t in (h, gu, dgu, hb):
            assert bool((t[none] == -7).all())
        for e, (a, b) in enumerate(segs):
            if a == b or any(a < d and s < b for i, (s, d) in enumerate(segs) if i != e):
                continue
            one = dict(off=torch.tensor([0, b - a], dtype=torch.int32, device=DEV), w=c["w"][e:e + 1], down=c["down"][e:e + 1],
                       **{n: c[n][a:b] for n in ("x", "dy", "gu")})
            glu._check_forward((h[a:b], gu[a:b]), one, "silu")
            glu._check_backward((dgu[a:b], hb[a:b]), one, "silu")
