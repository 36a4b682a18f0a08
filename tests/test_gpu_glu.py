"""The experts' gated unit (moe_grouped_glu) and its gradient
(moe_grouped_glu_backward) against plain loops over the segments in 64 bits.

Tolerance of the forward pass: g and u are sums of H exact products in fp32,
each within d = (H + 1) 2^-23 sum |a||b| (test_gpu_grouped.py).  Both
activations have |act'| <= 1.13, so h = act(g) u moves by at most
1.13 dg (|u| + du) + |act(g)| du; evaluating the activation in fp32 costs a
few steps of 2^-24 relative to q = g (c0 + c1 g^2) inside the exponential,
which |q| s (1 - s) <= 0.28 keeps below 2^-20 of |g u| all told.  A result
rounded to bf16 is off by at most half a step more, 2^-8 of its magnitude.

Of the backward pass: dh as such a sum over H, times u act' or act; act' in
fp32 within 2^-19 (its terms are at most 1.5 in magnitude, and q' stays below
200 for |g| <= 16); bf16 results."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
ACTS = ["silu", "gelu"]


def _case(counts, I, H, seed=0, lead=0, trail=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    R, E = lead + sum(counts) + trail, len(counts)
    off = lead + np.concatenate([[0], np.cumsum(counts)])
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    s = lambda n: 1.5 * n ** -0.5  # noqa: E731
    return dict(off=torch.from_numpy(off.astype(np.int32)).to(DEV), x=r(R, H), w=(r(E, 2 * I, H) * s(H)).to(torch.bfloat16),
                dy=r(R, H), down=(r(E, H, I) * s(H)).to(torch.bfloat16), gu=(r(R, 2 * I) * 2).to(torch.bfloat16))


def _act(g, act):
    """The activation and its derivative in 64 bits, by their textbook forms."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _half(y):
    return 2.0 ** -8 * y.abs()


def _forward(c, act):
    """-> (h, its tolerance in fp32, gu, its tolerance in fp32); rows of no segment stay 0."""
    off, x, w = c["off"].tolist(), c["x"].double(), c["w"].double()
    R, I = x.shape[0], w.shape[1] // 2
    gu, mag = (torch.zeros((R, 2 * I), dtype=torch.float64, device=DEV) for _ in range(2))
    for e in range(w.shape[0]):
        s = slice(off[e], off[e + 1])
        gu[s], mag[s] = x[s] @ w[e].T, x[s].abs() @ w[e].abs().T
    d = (x.shape[1] + 1) * 2.0 ** -23 * mag
    g, u, dg, du = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
    a, _ = _act(g, act)
    return a * u, 1.13 * dg * (u.abs() + du) + a.abs() * du + 2.0 ** -20 * (g * u).abs(), gu, d


def _backward(c, act):
    """-> [(dg, tolerance), (du, ...), (h, ...)], bf16's half step included."""
    off, dy, down, gu = c["off"].tolist(), c["dy"].double(), c["down"].double(), c["gu"].double()
    I = down.shape[2]
    dh, mag = (torch.zeros((dy.shape[0], I), dtype=torch.float64, device=DEV) for _ in range(2))
    for e in range(down.shape[0]):
        s = slice(off[e], off[e + 1])
        dh[s], mag[s] = dy[s] @ down[e], dy[s].abs() @ down[e].abs()
    d = (dy.shape[1] + 1) * 2.0 ** -23 * mag
    g, u = gu[:, :I], gu[:, I:]
    a, da = _act(g, act)
    out = []
    for v, t in ((dh * u * da, d * (u * da).abs() + 2.0 ** -19 * ((dh.abs() + d) * u.abs())),
                 (dh * a, d * a.abs() + 2.0 ** -20 * ((dh.abs() + d) * g.abs())), (a * u, 2.0 ** -20 * (g * u).abs())):
        out.append((v, t + _half(v.abs() + t)))
    return out


def _near(got, want, tol, rows=slice(None)):
    d = (got[rows].double() - want[rows]).abs()
    assert bool((d <= tol[rows] + 1e-37).all()), float((d / (tol[rows] + 1e-37)).max())


def _check_forward(got, c, act, rows=slice(None)):
    h, gu = got
    want, tol, pre, d = _forward(c, act)
    _near(h, want, tol if h.dtype == torch.float32 else tol + _half(want.abs() + tol), rows)
    _near(gu, pre, d + _half(pre.abs() + d), rows)


def _check_backward(got, c, act, rows=slice(None)):
    dgu, h = got
    I = h.shape[1]
    for t, (want, tol) in zip((dgu[:, :I], dgu[:, I:], h), _backward(c, act)):
        _near(t, want, tol, rows)


# few rows (the row-at-a-time kernel), single tiles, several tiles with ragged
# ends, and enough rows a segment for the paired tiles; widths that end inside
# a tile, inside a warp's sixteen outputs, and whole ones
SHAPES = [
    ([1], 8, 8),
    ([0, 2, 0, 0, 1, 0], 768, 2048),
    ([5, 0, 9], 40, 2056),
    ([33], 8, 72),
    ([1, 0, 40, 31, 0, 130], 264, 200),
    ([33] * 40, 136, 72),
    ([257, 0, 3, 190], 520, 264),
    ([700], 128, 512),
    ([300, 129, 513, 1], 392, 1000),
    ([0, 640, 129, 0, 500], 768, 136),
    ([260, 131], 72, 4104),
]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,I,H", SHAPES)
def test_forward_matches_64_bit_loops(cuda_lib, counts, I, H, dtype, act):
    c, st = _case(counts, I, H), cuda_lib.new_status()
    got = cuda_lib.grouped_glu(c["x"], c["w"], c["off"], act=act, keep=True, out_dtype=dtype, status=st)
    assert got[0].dtype == dtype and got[1].dtype == torch.bfloat16
    _check_forward(got, c, act)
    assert torch.equal(got[0], cuda_lib.grouped_glu(c["x"], c["w"], c["off"], act=act, out_dtype=dtype))
    assert int(st.item()) == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,I,H", SHAPES)
def test_backward_matches_64_bit_loops(cuda_lib, counts, I, H, act):
    c, st = _case(counts, I, H), cuda_lib.new_status()
    _check_backward(cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"], act=act, status=st), c, act)
    assert int(st.item()) == 0


@pytest.mark.parametrize("counts", [[2, 0, 3], [20, 0, 43, 1], [200, 0, 300]])
def test_rows_of_no_segment_are_left_as_they_were(cuda_lib, counts):
    c, n = _case(counts, 72, 136, lead=3, trail=5), sum(counts)
    new = lambda w: torch.full((n + 8, w), -7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    h, gu, dgu, hb = new(72), new(144), new(144), new(72)
    got = cuda_lib.grouped_glu(c["x"], c["w"], c["off"], out=h, gu=gu)
    assert got[0] is h and got[1] is gu
    _check_forward(got, c, "silu", slice(3, 3 + n))
    _check_backward(cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"], dgu=dgu, h=hb), c, "silu",
                    slice(3, 3 + n))
    for t in (h, gu, dgu, hb):
        assert bool((t[:3] == -7).all()) and bool((t[3 + n:] == -7).all())


@pytest.mark.parametrize("counts", [[2, 0, 1], [17, 0, 21, 30], [150, 0, 290, 141]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row_and_expert(cuda_lib, counts, bad):
    c = _case(counts, 72, 136)
    first = int(c["off"][-2])
    clean = {k: t.clone() for k, t in c.items()}
    c["x"][first:], c["dy"][first:], c["gu"][first:] = bad, bad, bad
    c["w"][1], c["down"][1] = bad, bad
    got = cuda_lib.grouped_glu(c["x"], c["w"], c["off"], keep=True)
    _check_forward(got, clean, "silu", slice(0, first))
    assert not bool(torch.isfinite(got[0][first:]).any())
    got = cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"])
    _check_backward(got, clean, "silu", slice(0, first))
    assert not bool(torch.isfinite(got[0][first:]).any())


@pytest.mark.parametrize("act", ACTS)
def test_activations_far_out(cuda_lib, act):
    """g from underflow to where its square overflows: act(g) is g or (a
    signed) zero there, and act' is 1 or 0, never NaN.  One product with 1
    makes g and u exact."""
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 90.0, -90.0, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38], device=DEV)
    n = 16
    x = torch.zeros((n, 8), dtype=torch.bfloat16, device=DEV)
    x[:len(g), 0] = g.to(torch.bfloat16)
    x[:, 1] = 1
    w = torch.zeros((1, 16, 8), dtype=torch.bfloat16, device=DEV)
    w[0, :8, 0], w[0, 8:, 1] = 1, 0.5  # g = x[0], u = 0.5
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    for rep in (1, 4):  # the row-at-a-time kernel, tiles
        xs, o = x.repeat(rep, 1), off * rep
        h = cuda_lib.grouped_glu(xs, w, o, act=act, out_dtype=torch.float32)
        a, da = _act(xs[:, :1].double(), act)
        ok = xs[:, :1].double().abs() < 50
        want = torch.where(ok, a, torch.where(xs[:, :1] > 0, xs[:, :1].double(), 0.0)) * 0.5
        _near(h, want.expand_as(h), 2.0 ** -19 * want.abs().expand_as(h) + 1e-18)
        dy = torch.zeros((n * rep, 8), dtype=torch.bfloat16, device=DEV)
        dy[:, 0] = 1
        down = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device=DEV)
        down[0, 0] = 1  # dh = 1
        gu = torch.cat([xs[:, :1].expand(-1, 8), torch.full_like(xs, 0.5)], 1).contiguous()
        dgu, _ = cuda_lib.grouped_glu_backward(dy, down, gu, o, act=act)
        want = torch.where(ok, da, (xs[:, :1] > 0).double()) * 0.5
        _near(dgu[:, :8], want.expand(-1, 8), (2.0 ** -8 * want.abs() + 2.0 ** -19).expand(-1, 8))


@pytest.mark.parametrize("counts", [[3, 1], [30, 50, 0, 11], [400, 0, 250]])
def test_bit_for_bit_again_captured_and_on_another_stream(cuda_lib, counts):
    c = _case(counts, 264, 200)
    call = lambda **kw: (cuda_lib.grouped_glu(c["x"], c["w"], c["off"], keep=True, **kw)  # noqa: E731
                         + cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"], **kw))
    first = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = call(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    # other segment sizes at replay: the launch does not depend on them
    keep = c["off"].clone()
    c["off"][1:-1] //= 2
    for t in out:
        t.fill_(-1)
    g.replay()
    torch.cuda.synchronize()
    _check_forward(out[:2], c, "silu")
    _check_backward(out[2:], c, "silu")
    c["off"].copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


@pytest.mark.parametrize("rows", [6, 60, 600])
@pytest.mark.parametrize("offsets", [[0, 4, 2, 6], [-1, 2, 3, 6], [0, 2, 3, 7], [0, 2 ** 31 - 1, 2, 6]])
def test_bad_offsets_leave_their_segment_out(cuda_lib, offsets, rows):
    scale = rows // 6
    off = torch.tensor([o if abs(o) > 9 else o * scale for o in offsets], dtype=torch.int32, device=DEV)
    c = _case([rows, 0, 0], 40, 72)
    for call in (lambda st: cuda_lib.grouped_glu(c["x"], c["w"], off, status=st),
                 lambda st: cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], off, status=st)):
        st = cuda_lib.new_status()
        call(st)
        assert int(st.item()) == cuda_lib.MOE_DEV_BAD_OFFSETS


def test_no_rows(cuda_lib):
    c = _case([4, 0], 40, 72)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert cuda_lib.grouped_glu(c["x"][:0], c["w"], off).shape == (0, 40)
    dgu, h = cuda_lib.grouped_glu_backward(c["dy"][:0], c["down"], c["gu"][:0], off)
    assert dgu.shape == (0, 80) and h.shape == (0, 40)


def test_gradients_against_differences(cuda_lib):
    """The block's loss sum(y dy), y = down h, moved along a direction of g and
    u: central differences in 64 bits of the formulas, the step 2^-10, against
    the kernel's dgu.  The third derivative's term is below 2^-20 of the
    magnitudes; dgu is off by half a bf16 step an element, independently."""
    c = _case([30, 0, 140], 136, 264)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    v = torch.randn(c["gu"].shape, generator=gen, device=DEV, dtype=torch.float64)
    off, I = c["off"].tolist(), 136

    def loss(gu, act):
        h = _act(gu[:, :I], act)[0] * gu[:, I:]
        return sum(((h[a:b] @ c["down"][e].double().T) * c["dy"][a:b].double()).sum()
                   for e, (a, b) in enumerate(zip(off, off[1:])))

    for act in ACTS:
        dgu, _ = cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"], act=act)
        gu, t = c["gu"].double(), 2.0 ** -10
        num = (loss(gu + t * v, act) - loss(gu - t * v, act)) / (2 * t)
        m = (dgu.double() * v).abs()
        # (independent half steps: four deviations of their sum)
        tol = 4 * 2.0 ** -8 * float((m * m).sum().sqrt()) + 2.0 ** -16 * float(m.sum())
        assert abs(float(num - (dgu.double() * v).sum())) <= tol


def _largest(cuda_lib, R, I, H, E, off, rows):
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, w, o = r(R, H), r(E, 2 * I, H) * H ** -0.5, off.tolist()
    h, gu = cuda_lib.grouped_glu(x, w, off, keep=True)
    down = (w.view(-1)[:E * H * I]).view(E, H, I)
    dgu, hb = cuda_lib.grouped_glu_backward(x, down, gu, off)
    for at in rows:
        e = next(i for i in range(E) if o[i] <= at < o[i + 1])
        one = lambda t: t[at:at + 1].contiguous()  # noqa: E731
        c = dict(off=torch.tensor([0, 1], dtype=torch.int32, device=DEV), x=one(x), w=w[e:e + 1], dy=one(x),
                 down=down[e:e + 1], gu=one(gu))
        _check_forward((one(h), one(gu)), c, "silu")
        _check_backward((one(dgu), one(hb)), c, "silu")


def test_offsets_past_32_bits(cuda_lib):
    R = 1_100_000
    off = torch.tensor([0, 1_000_000, 1_000_000, R], dtype=torch.int32, device=DEV)
    _largest(cuda_lib, R, 2048, 64, 3, off, (0, 999_999, 1_000_000, 1_060_000, R - 1))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_the_largest_matrices(cuda_lib, rows):
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    _largest(cuda_lib, rows, cuda_lib.MAX_DIM, cuda_lib.MAX_DIM, 1, off, (0, rows - 1))
    torch.cuda.empty_cache()


def test_the_most_rows_and_segments(cuda_lib):
    R, E = cuda_lib.MAX_ROWS, cuda_lib.MAX_E
    off = (torch.arange(E + 1, dtype=torch.int64) * 16363).clamp(max=R).to(torch.int32)
    off[-1] = R
    _largest(cuda_lib, R, 40, 72, E, off.to(DEV), (0, 16362, 16363, R - 1))


def test_two_streams_at_once(cuda_lib):
    cases = [_case(n, 264, 200, seed=i) for i, n in enumerate(([3, 1], [30, 50, 0, 11], [400, 0, 250]))]
    call = lambda c, **kw: (cuda_lib.grouped_glu(c["x"], c["w"], c["off"], keep=True, **kw)  # noqa: E731
                            + cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"], **kw))
    want = [call(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [call(c, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
