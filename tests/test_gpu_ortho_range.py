"""Orthogonalisation (moe_orthogonalize) at its largest sizes, and what it loses
where that would show most."""
import math

import pytest
import torch

import test_gpu_ortho as ortho

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("N,K", [(16384, 16256), (16384, 16258), (16383, 16257), (16383, 16259)])
@pytest.mark.parametrize("v", [0.7, 1.45, 1.1, 0.9])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_norm_of_many_equal_values(cuda_lib, N, K, v, dtype):
    """X = G / |G|_F alone: 1 / sqrt(N K) in bf16, whatever the value.  The
    sizes put it 2.3e-5 above or 3.8e-5 below the middle of two bf16 values, so
    that a norm which a long sum of squares left off by more shows up in every
    value of the result.  Allowed is 2^-17 = 7.6e-6: 2^-19 of the norm and
    half of fp16's smallest step, 2^-25, in what 22 bits leave of 2^-6."""
    g = torch.full((N, K), v, device=DEV).to(dtype)
    want = 1.0 / math.sqrt(N * K)
    got = cuda_lib.orthogonalize(g, steps=1, coeffs=(1.0, 0.0, 0.0), eps=0.0)
    lo, hi = (torch.tensor(want * (1 + s * 2.0 ** -17), dtype=torch.float64).to(BF16) for s in (-1, 1))
    assert bool(lo == hi)
    assert bool((got == lo.to(DEV)).all()), (float(got[0, 0]), float(lo))
    del g, got
    torch.cuda.empty_cache()


def _both_halves(g):
    """The recurrence of five steps with the kernel's roundings, X in two fp16 values into the last step too."""
    (a, b, c), r = ortho.NS, lambda t, s: (t * s).half().double() / s
    two = lambda t: r(t, ortho.UP) + r(t - r(t, ortho.UP), ortho.UP)  # noqa: E731
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = two(x / (x.flatten(-2).norm(dim=-1).view(-1, 1, 1) + 1e-7))
    for i in range(5):
        s = 0.5 if i >= 3 else 0.0
        h = r(x, ortho.UP)
        m = r(h @ h.mT - s * torch.eye(x.shape[-2], dtype=torch.float64, device=DEV), 1.0)
        x = (a + b * s + c * s * s) * x + r((b + 2 * c * s) * m + c * (m @ m), 1.0) @ h
        x = two(x) if i < 4 else x
    return x.mT if tall else x


@pytest.mark.parametrize("N,K,rank", [(256, 256, 24), (500, 130, 1)])
def test_few_directions_keep_both_halves(cuda_lib, N, K, rank):
    """In the directions that G lacks every step enlarges what was rounded off
    X by a = 3.4, the last one too.  The kernel's distance from the exact
    result is that of the recurrence with its roundings and the result's own to
    bf16, which are independent of it: squares add.  Sums of 2 10^5 or more
    independent errors scatter by 0.2 %; allowed are 2 %."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    g = r(4, N, rank) @ r(4, rank, K)
    want = ortho._recurrence(g, 5, ortho.NS, 1e-7, False)
    own, lost = (want.to(BF16).double() - want).norm(), (_both_halves(g) - want).norm()
    off = (cuda_lib.orthogonalize(g).double() - want).norm()
    assert float(off) <= 1.02 * math.hypot(float(own), float(lost)), float(off) / math.hypot(float(own), float(lost))


@pytest.mark.parametrize("N,K", [(3100, 4097), (4100, 2800)])
def test_long_short_sides_match_64_bits(cuda_lib, N, K):
    g = ortho._g(1, N, K)
    ortho._check(cuda_lib.orthogonalize(g), g)


@pytest.mark.parametrize("a,b", [((128, 128), (128, 128)), ((128, 120), (128, 100)), ((90, 128), (100, 128))])
def test_the_largest_matrices(cuda_lib, a, b):
    """Kronecker products A x B: their singular vectors are those of A and B,
    their singular values all products, so that the exact result follows from
    the recurrence of a number.

    Tolerance: at most 12.2 half steps of fp16 a step and four steps that count
    (test_gpu_ortho.py), evenly spread, which over 10^8 values is 3^-1/2 of
    that in 2-norm; and half a step of bf16, likewise."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    A, B = (torch.randn(s, generator=gen, device=DEV, dtype=torch.float64) for s in (a, b))
    g = torch.kron(A, B).float().contiguous()
    (ua, sa, va), (ub, sb, vb) = (torch.linalg.svd(t, full_matrices=False) for t in (A, B))
    s = sa.unsqueeze(1) * sb.unsqueeze(0)
    s = s / (s.norm() + 1e-7)
    c0, c1, c2 = ortho.NS
    for _ in range(5):
        s = s * (c0 + s * s * (c1 + c2 * s * s))
    got = cuda_lib.orthogonalize(g)
    del g
    off = size = 0.0
    for i in range(a[0]):  # the rows that A's i-th row makes
        t = torch.einsum("p,qr,pr,pm->mqr", ua[i], ub, s, va)  # [A's columns, B's rows, B's directions]
        want = (t @ vb).transpose(0, 1).reshape(b[0], -1)
        off += float((got[i * b[0]:(i + 1) * b[0]].double() - want).square().sum())
        size += float(want.square().sum())
    tol = (4 * 12.2 * 2.0 ** -12 + 2.0 ** -8) / 3 ** 0.5
    assert math.sqrt(off / size) <= tol, math.sqrt(off / size)
    torch.cuda.empty_cache()
