"""Orthogonalised matrices (moe_orthogonalize) against the same recurrence in
64 bits.

Tolerance: the kernel rounds X (which it carries in two fp16 values, into the
last step in one), A' = X X^T
(in the last two steps less 1/2) and B, what b A + c A A then comes to, to fp16
for its products, half a step (2^-12) a value; with a short side of up to 96 it
rounds X alone, and for X X^T alone.  How far that carries depends on the
matrix, so the recurrence is also run in 64 bits with these roundings, and its
distance from the exact one is counted twice (once for the roundings, once for
those that the fp32 sums decide the other way).  It has to stay below 2^-6 of
the result itself, what one value a matrix may come to, where nothing averages.
With X' / X at least 0.68, |A| at most 1.3, |B| at most 2.85 (b^2 / 4c) and
|A (b + 2 c A)| at most 0.85, 2^-12 of X count 2 * 0.85 / 0.68 times through A
and 2.85 / 0.68 times through B X, those of A 0.85 / 0.68 and those of B 2.85 /
0.68 times: 12.2 2^-12 a step, below 2^-8; four of five steps deal with values
that large, each passing on what came before at most as it is.  Values of X
below fp16's normal ones are off by up to 2^-25 absolutely, 2^-33 of X without
its factor 2^8, and a step enlarges what is that small by |a| at most: sqrt(N K)
2^-33 (1 + |a|)^steps of 2-norm beside the rest, which counts where eps is all
that a matrix is divided by.  The result's own rounding to bf16 adds half a
step, 2^-8 of each value.  Distances are 2-norms of whole matrices."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
NS = (3.4445, -4.7750, 2.0315)
UP = 256.0  # the factor that X carries


def _recurrence(g, steps, coeffs, eps, half):
    r = (lambda t, s: (t * s).half().double() / s) if half else (lambda t, s: t)
    two = lambda t: r(t, UP) + r(t - r(t, UP), UP) if half else t  # noqa: E731
    a, b, c = coeffs
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = two(x / (x.flatten(-2).norm(dim=-1).view(*x.shape[:-2], 1, 1) + eps))
    # (a short side's A and B are held in 22 bits, and X rounded for X X^T alone: exact here but for that)
    short = x.shape[-2] <= 96
    for i in range(steps):
        s = 0.5 if steps - i <= 2 and not short else 0.0
        h = r(x, UP)
        if half and short:
            m = h @ h.mT
            x = two(a * x + (b * m + c * (m @ m)) @ x)
            continue
        m = r(h @ h.mT - s * torch.eye(x.shape[-2], dtype=torch.float64, device=DEV), 1.0)
        x = (a + b * s + c * s * s) * x + r((b + 2 * c * s) * m + c * (m @ m), 1.0) @ h
        x = x if i + 1 == steps or not half else r(x, UP) if i + 2 == steps else two(x)
    return x.mT if tall else x


def _check(got, g, steps=5, coeffs=NS, eps=1e-7):
    assert got.shape == g.shape and got.dtype == torch.bfloat16
    norm = lambda t: t.flatten(-2).norm(dim=-1)  # noqa: E731
    want = _recurrence(g, steps, coeffs, eps, False)
    lost = norm(_recurrence(g, steps, coeffs, eps, True) - want)
    tiny = (g.shape[-1] * g.shape[-2]) ** 0.5 * 2.0 ** -33 * (1 + abs(coeffs[0])) ** steps
    assert bool((lost <= 2.0 ** -6 * norm(want) + tiny).all()), float((lost / norm(want)).max())
    off = norm(got.double() - want)
    tol = 2.0 ** -8 * norm(want) + 2 * lost + 2.0 ** -40
    assert bool((off <= tol).all()), float((off / tol).max())


def _g(E, N, K, dtype=torch.float32, seed=0, sigma=1e-3):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    g = (r(E, N, K) + 0.1 * r(E, N, 2) @ r(E, 2, K)) * sigma
    return (g if E > 1 else g[0]).to(dtype)


# one value, vectors, odd sizes both ways up, ends inside tiles, enough tiles
# for pairs of CTAs, contractions of several accumulators
SHAPES = [(1, 1, 1), (1, 1, 40), (1, 33, 1), (3, 2, 5), (1, 8, 64), (2, 65, 63), (5, 130, 257), (4, 257, 131), (1, 515, 390),
          (3, 96, 200), (3, 200, 97), (64, 90, 100), (90, 264, 300), (40, 300, 520), (80, 520, 128), (256, 16, 24), (2, 72, 3001), (3, 1100, 1201)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,N,K", SHAPES)
def test_matches_the_recurrence_in_64_bits(cuda_lib, E, N, K, dtype):
    g, st = _g(E, N, K, dtype), cuda_lib.new_status()
    _check(cuda_lib.orthogonalize(g, status=st), g)
    assert int(st.item()) == 0


@pytest.mark.parametrize("N,K,rank", [(256, 256, 24), (256, 1000, 8), (500, 130, 1), (70, 70, 3)])
def test_few_directions(cuda_lib, N, K, rank):
    """The gradient of a few tokens: what is rounded off in the directions that
    it lacks must not grow into the result."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    g = r(3, N, rank) @ r(3, rank, K)
    _check(cuda_lib.orthogonalize(g), g)


@pytest.mark.parametrize("N,K", [(40, 72), (200, 72), (300, 300)])
@pytest.mark.parametrize("steps,coeffs", [(1, NS), (2, NS), (16, (2.0, -1.5, 0.5)), (3, (1.5, -0.5, 0.0)), (4, (0.0, 1.0, 0.0))])
def test_steps_and_coefficients(cuda_lib, N, K, steps, coeffs):
    g = _g(3, N, K)
    _check(cuda_lib.orthogonalize(g, steps=steps, coeffs=coeffs), g, steps, coeffs)


def test_rows_become_orthonormal(cuda_lib):
    """Steps that converge leave X X^T = 1, up to the result's rounding: two
    bf16 roundings of 2^-8 a value and fp16's 2^-12 ones, in 2-norm of the
    matrix below 2^-7 |1|_F."""
    g = _g(4, 72, 500, sigma=1.0)
    x = cuda_lib.orthogonalize(g, steps=14, coeffs=(2.0, -1.5, 0.5)).double()
    one = torch.eye(72, dtype=torch.float64, device=DEV)
    assert float((x @ x.mT - one).flatten(1).norm(dim=1).max()) <= 2.0 ** -7 * 72 ** 0.5


@pytest.mark.parametrize("N,K", [(64, 96), (131, 70)])
def test_any_magnitude(cuda_lib, N, K):
    """Scaled by powers of two that overflow or underflow a sum of squares,
    the result is the same bit for bit (without eps)."""
    g = _g(2, N, K, sigma=1.0)
    want = cuda_lib.orthogonalize(g, eps=0.0)
    for p in (-110, -60, 60, 110):
        assert torch.equal(cuda_lib.orthogonalize(g * 2.0 ** p, eps=0.0), want), p
    # beside eps a tiny matrix shrinks instead
    small = g * 2.0 ** -60
    _check(cuda_lib.orthogonalize(small, eps=1.0), small, eps=1.0)


def test_zero_matrices_and_what_is_not_finite(cuda_lib):
    g = _g(6, 100, 130)
    want = cuda_lib.orthogonalize(g)
    g[1] = 0
    g[3, 5, 7] = float("nan")
    g[4, 99, 0] = float("inf")
    got = cuda_lib.orthogonalize(g)
    assert bool((got[1] == 0).all())
    assert bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[4]).all())
    for i in (0, 2, 5):
        assert torch.equal(got[i], want[i])
    assert bool(torch.isnan(cuda_lib.orthogonalize(torch.zeros_like(g), eps=0.0)).all())


@pytest.mark.parametrize("E,N,K", [(1, 40, 72), (7, 260, 130), (90, 264, 300)])
def test_in_place_captured_and_on_another_stream(cuda_lib, E, N, K):
    g = _g(E, N, K, torch.bfloat16)
    first = cuda_lib.orthogonalize(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = cuda_lib.orthogonalize(g, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cuda_lib.orthogonalize(g)
    keep = g.clone()
    g.copy_(_g(E, N, K, torch.bfloat16, seed=9))
    graph.replay()
    torch.cuda.synchronize()
    _check(out, g)
    g.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    assert cuda_lib.orthogonalize(g, out=g) is g and torch.equal(g, first)


def test_two_streams_at_once(cuda_lib):
    cases = [_g(*s, seed=i) for i, s in enumerate(((1, 40, 72), (7, 260, 130), (90, 264, 300)))]
    want = [cuda_lib.orthogonalize(g) for g in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [cuda_lib.orthogonalize(g, stream=s) for g, s in zip(cases, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("N,K", [(24, 16384), (16384, 24)])
def test_the_longest_side(cuda_lib, N, K):
    g = _g(2, N, K)
    _check(cuda_lib.orthogonalize(g), g)


def test_offsets_past_32_bits(cuda_lib):
    """More than 2^31 values: the last matrices of the batch are those of a small one."""
    E, N, K = 140, 2040, 8192
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    g = torch.randn((E, N, K), generator=gen, device=DEV, dtype=torch.bfloat16)
    got = cuda_lib.orthogonalize(g, steps=1)
    for e in (0, E - 1):
        _check(got[e], g[e], steps=1)
    torch.cuda.empty_cache()
