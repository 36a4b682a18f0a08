"""Long sums of the grouped products: what the tensor cores' truncating
additions take from them stays bounded, however long the sum and whatever the
result's type.

An accumulator takes 64 additions (of 16 terms each).  An addition that
truncates takes less than a step, 2^-23, of the running sum, which in a sum of
one sign is half of the part's on average: 64 / 2 * 2^-23 = 2^-18.  The parts
are added with rounding to nearest, whose errors have either sign.  Sums of
random signs lose no more of their 2-norm.  One accumulator for all terms
loses 7.4e-5 of 16384 terms of one sign, and 1.9e-5 of those of random signs.

The cases are such that the weight gradients' rows are not cut into parts of
their own (at least 39 paired or 77 single tiles on 152 SMs)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOST = 2.0 ** -18

CASES = [
    ("fwd", [512], 2048, 16384),                       # paired tiles
    ("fwd", [60], 2048, 16384),                        # single tiles
    ("fwd", [500, 0, 300], 1024, 2056),                # three parts, the last of one step
    ("dx", [512], 32768, 2048),
    ("dx", [60], 32768, 2048),
    ("dw", [1 << 18], 1792, 1792),
    ("dw", [5, 0, 1 << 17, 33, 700], 1792, 1792),      # one segment holds nearly all rows
    ("dw", [1 << 17], 10240, 128),
]


def _inputs(op, counts, N, K, one_sign, seed=0):
    """x, w, dy; of one sign: uniform in [0.5, 1.5), times scales that spread
    the results over two binades (so that roundings to bf16 fall evenly)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def draw(*shape):
        return torch.rand(shape, generator=g, device=DEV) + 0.5 if one_sign else torch.randn(shape, generator=g, device=DEV)

    def spread(t, dim):
        if one_sign:
            t *= (2.0 ** torch.linspace(0, 1, t.shape[dim], device=DEV)).view([-1 if d == dim % t.dim() else 1 for d in range(t.dim())])
        return t.to(torch.bfloat16)

    R, E = sum(counts), len(counts)
    if op == "fwd":
        return spread(draw(R, K), 0), spread(draw(E, N, K), 1), None
    if op == "dx":
        return None, spread(draw(E, N, K), 2), spread(draw(R, N), 0)
    return spread(draw(R, K), 1), None, spread(draw(R, N), 1)


def _result_and_reference(api, op, counts, x, w, dy, dtype):
    """-> (values, 64-bit values); dw: 128 rows and columns at both ends of the longest segment's matrix."""
    off = torch.tensor([0, *counts], device=DEV).cumsum(0).to(torch.int32)
    segs = [slice(int(a), int(b)) for a, b in zip(off[:-1], off[1:])]
    if op == "fwd":
        y = api.grouped_gemm(x, w, off, out_dtype=dtype)
        return y.double(), torch.cat([x[s].double() @ w[e].double().T for e, s in enumerate(segs)])
    if op == "dx":
        y = api.grouped_gemm_dx(dy, w, off, out_dtype=dtype)
        return y.double(), torch.cat([dy[s].double() @ w[e].double() for e, s in enumerate(segs)])
    e = max(range(len(counts)), key=counts.__getitem__)
    y = api.grouped_gemm_dw(dy, x, off, out_dtype=dtype)[e]
    ends = lambda t, d: torch.cat([t.narrow(d, 0, min(128, t.shape[d] // 2)),  # noqa: E731
                                   t.narrow(d, t.shape[d] - min(128, t.shape[d] // 2), min(128, t.shape[d] // 2))], d)
    return ends(ends(y, 0), 1).double(), ends(dy[segs[e]], 1).double().T @ ends(x[segs[e]], 1).double()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("op,counts,N,K", CASES)
def test_long_sums_of_one_sign_do_not_shrink(cuda_lib, op, counts, N, K, dtype):
    """The mean relative error, a bias and no scatter.  A rounding to bf16 adds
    an error of at most 2^-8, evenly spread: 2^-8 / sqrt(3) at most from one
    result, of their mean that over sqrt(n); five times that is allowed."""
    got, ref = _result_and_reference(cuda_lib, op, counts, *_inputs(op, counts, N, K, True), dtype)
    bias = float((got / ref - 1).mean())
    assert abs(bias) <= LOST + (5 * 2.0 ** -8 / (3 * ref.numel()) ** 0.5 if dtype == torch.bfloat16 else 0)


@pytest.mark.parametrize("op,counts,N,K", CASES)
def test_long_sums_of_random_signs(cuda_lib, op, counts, N, K):
    got, ref = _result_and_reference(cuda_lib, op, counts, *_inputs(op, counts, N, K, False), torch.float32)
    assert float((got - ref).norm() / ref.norm()) <= LOST
