"""The grouped products' paired tiles (two CTAs on one tile) where segments
are many and widely unequal, and their ends ragged."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(counts, N, K, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
    R = sum(counts)
    return off, r(R, K), (r(len(counts), N, K) * 0.05).to(torch.bfloat16), r(R, N)


def _call(api, op, off, x, w, dy, dtype):
    if op == "fwd":
        return api.grouped_gemm(x, w, off, out_dtype=dtype)
    if op == "dx":
        return api.grouped_gemm_dx(dy, w, off, out_dtype=dtype)
    return api.grouped_gemm_dw(dy, x, off, out_dtype=dtype)


def _check(op, got, off, x, w, dy, segments):
    """got against 64 bits at the given segments: (terms + 1) additions of at
    most a step, 2^-23, of the sum of magnitudes each, and half a step, 2^-8,
    of a bf16 result."""
    o = off.tolist()
    for e in segments:
        s = slice(o[e], o[e + 1])
        a, b = {"fwd": (x[s], w[e].T), "dx": (dy[s], w[e]), "dw": (dy[s].T, x[s])}[op]
        y, m, terms = a.double() @ b.double(), a.double().abs() @ b.double().abs(), a.shape[1]
        tol = (terms + 1) * 2.0 ** -23 * m
        if got.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (y.abs() + tol)
        d = (got[e if op == "dw" else s].double() - y).abs()
        assert bool((d <= tol).all()), (e, float((d / tol.clamp(min=1e-300)).max()))


# every residue of a segment's end modulo the 16 rows of an MMA and the 64 of a stage
RAGGED = [430 + 37 * i % 129 for i in range(40)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_behind_a_segment_do_not_reach_its_gradient(cuda_lib, bad, dtype):
    """Every other segment's rows are not finite: the gradients between them
    are those of their own rows, although their last MMAs reach into those
    rows, which each CTA of a pair clears in its own shared memory."""
    off, x, w, dy = _case(RAGGED, 520, 392)
    for e in range(1, len(RAGGED), 2):
        s = slice(int(off[e]), int(off[e + 1]))
        x[s], dy[s] = bad, bad
    first = None
    for _ in range(10):
        got = cuda_lib.grouped_gemm_dw(dy, x, off, out_dtype=dtype)
        if first is None:
            first = got
            _check("dw", got, off, x, w, dy, range(0, len(RAGGED), 2))
            assert not bool(torch.isfinite(got[1::2]).any())
        assert torch.equal(got[0::2], first[0::2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_many_widely_unequal_segments(cuda_lib, op, dtype):
    """Paired tiles over segments from no row to thousands."""
    g = np.random.default_rng(0)
    counts = [int(c) for c in 40000 * g.permutation(np.arange(1, 61) ** -1.5 / np.sum(np.arange(1, 61) ** -1.5))]
    counts[7] = counts[30] = 0
    counts[3] = 1
    assert sum(counts) >= 384 * len(counts) and min(counts) == 0 and max(counts) > 10000
    off, x, w, dy = _case(counts, 392, 520)
    st = cuda_lib.new_status()
    got = _call(cuda_lib, op, off, x, w, dy, dtype)
    _check(op, got, off, x, w, dy, range(len(counts)))
    assert int(st.item()) == 0
