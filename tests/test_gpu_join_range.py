"""Where the join's gradients could leave fp32's range or precision although
their results do not: rows of any magnitude, an eps next to nothing, an eps of
nothing with rows of nothing, and column sums over many tokens.

Tolerances and formulas as in test_gpu_join.py, where not said otherwise."""
import pytest
import torch

import test_gpu_join as join

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("dx", "do", "dw", "dpost", "dscale", "dpre")

# a vector a thread with its rows kept, and several, read again; blocks of several warps and of one
SHAPES = [(9, 3, 136), (70, 2, 2056), (5, 4, 8200)]


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("p,q", [(47, 0), (-47, 0), (0, 47), (0, -47), (47, -47), (-47, 47), (40, 40), (-40, -40)])
def test_rows_of_any_magnitude(cuda_lib, T, k, H, p, q):
    """Without eps the gradients of rows 2^p (the stream) and 2^q (the block's)
    times as large are the same bits times a power of two: all operations
    scale, as long as nothing leaves fp32's range.  Sums of squares reach
    2^(2 |p|) times e^8 H, below 2^120; a gradient 2^-(p + q) times a few
    2^-30, above 2^-120."""
    c = join._case(T, k, H, F32, F32, F32)
    c["eps"], c["dy"] = 0.0, None
    want = dict(zip(NAMES, join._call_back(cuda_lib, c)))
    c["x"], c["o"] = c["x"] * 2.0 ** p, c["o"] * 2.0 ** q
    got = dict(zip(NAMES, join._call_back(cuda_lib, c)))
    # dx ~ 1 / y; do ~ dx / o, dw ~ dx, dpost and dscale ~ dx (the norm takes o's magnitude away), dpre ~ 1
    for n, e in (("dx", -p), ("do", -p - q), ("dw", -p), ("dpost", -p), ("dscale", -p), ("dpre", 0)):
        assert bool(torch.isfinite(want[n]).all()) and torch.equal(got[n], want[n] * 2.0 ** e), n


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("p", [47, 30])
def test_large_rows_match_64_bits(cuda_lib, T, k, H, p):
    c = join._case(T, k, H, F32, F32, F32)
    c["x"], c["o"] = c["x"] * 2.0 ** p, c["o"] * 2.0 ** p
    join._check(join._call(cuda_lib, c), c)
    c["dy"] = c["dy"] * 2.0 ** -p  # (as large as the norm's part)
    join._check_back(join._call_back(cuda_lib, c), c)


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("eps", [1e-20, 1e-30, 1e-36])
def test_rows_of_zeros_beside_a_tiny_eps(cuda_lib, monkeypatch, T, k, H, eps):
    """1 / sqrt(eps) is within fp32's range, its cube is not; where a row is
    zero the cube counts for nothing.  dn is small, since dx is 1 / sqrt(eps)
    times as large."""
    monkeypatch.setattr(join, "EPS", float(torch.tensor(eps, dtype=F32)))
    c = join._case(T, k, H, F32, F32, F32)
    c["eps"], c["dn"] = eps, c["dn"] * eps ** 0.5
    c["o"][c["pos"][1].long()] = 0
    c["x"][2] = 0
    join._check(join._call(cuda_lib, c), c)
    join._check_back(join._call_back(cuda_lib, c), c)


@pytest.mark.parametrize("T,k,H", SHAPES)
def test_tokens_without_rows_and_without_eps(cuda_lib, monkeypatch, T, k, H):
    """A token whose routes are all dropped passes the stream on and adds
    nothing to the sums, with eps = 0 too (the norm of nothing is nothing)."""
    monkeypatch.setattr(join, "EPS", 0.0)
    c = join._case(T, k, H, F32, F32, F32)
    c["eps"] = 0.0
    c["pos"][1], c["pos"][T - 1] = -1, -1
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[1] = keep[T - 1] = False
    there = {n: c[n][keep].contiguous() for n in ("x", "dy", "dn", "pos", "w")}
    y, n = join._call(cuda_lib, c)
    assert torch.equal(y[~keep], c["x"][~keep])
    alone = cuda_lib.combine_norm(c["x"][~keep].contiguous(), pre=c["pre"], eps=0.0, n_dtype=F32)[1]
    assert torch.equal(n[~keep], alone)
    sub = {**c, **there}
    join._check((y[keep], n[keep]), sub)
    got, want = dict(zip(NAMES, join._call_back(cuda_lib, c))), join._backward(sub)
    for m in ("dpost", "dscale"):
        join._near(got[m], *want[m])
    join._near_rows(got["dx"][keep], *want["dx"])
    assert bool((got["dw"][~keep] == 0).all())
    stream = join._backward(dict(c, o=None))
    join._near(got["dpre"], *stream["dpre"])
    join._near_rows(got["dx"][~keep], *(t[~keep] for t in stream["dx"]))


@pytest.mark.parametrize("T,k,H", SHAPES)
def test_rows_of_zeros_without_eps(cuda_lib, T, k, H):
    """0 / 0 counts as 0: the norm of a row of zeros is zeros, and so is its gradient."""
    c = join._case(T, k, H, F32, F32, F32)
    c["eps"] = 0.0
    clean, back = join._call(cuda_lib, c), join._call_back(cuda_lib, c)
    rows = c["pos"][1].long()
    c["o"][rows] = 0
    c["x"][2] = 0
    c["x"][1] = 0
    y, n = join._call(cuda_lib, c)
    assert bool((y[1] == 0).all()) and bool((n[1] == 0).all()) and bool(torch.isfinite(n).all())
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[1] = keep[2] = False
    assert torch.equal(n[keep], clean[1][keep])
    got = join._call_back(cuda_lib, c)
    assert all(bool(torch.isfinite(t).all()) for t in got)
    assert torch.equal(got[0][1], c["dy"][1]) and torch.equal(got[0][2], c["dy"][2])
    assert bool((got[1][rows] == 0).all()) and bool((got[2][1] == 0).all())
    assert torch.equal(got[0][keep], back[0][keep]) and torch.equal(got[2][keep], back[2][keep])


def test_column_sums_over_many_tokens(cuda_lib):
    """2^20 tokens, all terms of a column alike and of one sign: a sum of n
    fp32 additions one after the other is off by up to n / 2 2^-24.  A block
    adds up 256 tokens at most before it puts them aside (2^20 / 152 / 256 = 27
    times on 152 SMs, 108 times for the most tokens), and the blocks' sums take
    28 more: (256 + 108 + 28) / 2 2^-24 < 2^-16.  The terms' own roundings,
    2^-20, count on top."""
    T, H = 1 << 20, 2056
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    r = lambda: (0.5 + torch.rand(H, generator=g, device=DEV))  # noqa: E731
    row = {n: r().to(BF16) for n in ("y", "dy", "dn", "o")}
    post, scale, pre = r(), r(), r()
    y, dy, dn, o = (row[n].expand(T, H).contiguous() for n in ("y", "dy", "dn", "o"))
    got = cuda_lib.combine_norm_backward(dy, dn, y, o, post=post, scale=scale, pre=pre, eps=1e-6)
    one = lambda t: t.double().view(1, H)  # noqa: E731
    a, ny = one(row["dn"]) * one(pre), join._rms(one(row["y"]))
    d = one(row["dy"]) + ny * a - one(row["y"]) * ny ** 3 * (a * one(row["y"])).mean()
    hat = one(row["o"]) * join._rms(one(row["o"]))
    want = (d * one(scale) * hat, d * hat * one(post), one(row["dn"]) * one(row["y"]) * ny)
    for n, t, w in zip(("dpost", "dscale", "dpre"), got[3:], want):
        off = float((t.double() / (T * w.flatten()) - 1).abs().max())
        assert off <= 2.0 ** -16 + 2.0 ** -20, (n, off)
    torch.cuda.empty_cache()


def test_a_scale_without_rows_counts_for_nothing(cuda_lib):
    """At the C entry, where the scale is a number beside the rows' pointer."""
    x = torch.randn((5, 72), device=DEV)
    pre = torch.ones(72, device=DEV)
    want = cuda_lib.combine_norm(x, pre=pre, n_dtype=F32)[1]
    n, st = torch.empty_like(x), torch.cuda.current_stream().cuda_stream
    for s in (float("inf"), float("nan"), 2.0):
        assert cuda_lib._lib.moe_combine_norm(x.data_ptr(), 0, None, 1, None, None, 5, 72, 0, 0, None, None, s, pre.data_ptr(),
                                              1e-6, None, n.data_ptr(), 0, None, st) == 0
        assert torch.equal(n, want)
