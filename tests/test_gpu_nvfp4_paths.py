"""NVFP4: the paired product where a row is no whole number of stages, and the
matrix quantiser with many more chunks than are in flight at once."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [32, 96, 448, 1312])
@pytest.mark.parametrize("counts,N", [([300, 0, 257], 520), ([129, 511, 0, 130, 1], 264)])
def test_paired_product_of_rows_that_end_inside_a_stage(cuda_lib, counts, N, K, dtype):
    """A stage is 256 elements; the scales of such rows are read from memory
    by the warps themselves.  K exact products are summed in fp32 with
    additions that may truncate, (K + 1) 2^-23 of the magnitudes' sum; two
    roundings by the scales, 2^-24 each; half a step 2^-8 of a bf16 result."""
    g = torch.Generator(device=DEV)
    g.manual_seed(K)
    R = sum(counts)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
    # magnitudes that differ from block to block: each has a scale of its own
    mag = lambda *s: torch.exp2(torch.randint(-3, 4, s, generator=g, device=DEV).float()).repeat_interleave(16, -1)  # noqa: E731
    x = torch.randn((R, K), generator=g, device=DEV) * mag(R, K // 16)
    w = torch.randn((len(counts), N, K), generator=g, device=DEV) * mag(len(counts), N, K // 16)
    xq, wq = cuda_lib.quantize_nvfp4(x), cuda_lib.quantize_nvfp4(w)
    out = torch.full((R, N), -7.0, dtype=dtype, device=DEV)
    st = cuda_lib.new_status()
    cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out=out, status=st)
    xv, wv = cuda_lib.dequantize_nvfp4(*xq).double(), cuda_lib.dequantize_nvfp4(*wq).double()
    for e in range(len(counts)):
        s = slice(int(off[e]), int(off[e + 1]))
        y, m = xv[s] @ wv[e].T, xv[s].abs() @ wv[e].abs().T
        tol = ((K + 1) * 2.0 ** -23 + 2 * 2.0 ** -24) * m
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (y.abs() + tol)
        assert bool(((out[s].double() - y).abs() <= tol).all()), e
    assert int(st.item()) == 0


def _nearest(a, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    t = torch.tensor(table, dtype=torch.float64, device=a.device)
    mid = (t[1:] + t[:-1]) / 2
    lo, hi = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127]


def _definition(x):
    """Matrices [G, rows, cols] -> (q, bs, gs), from the definition in 64 bits."""
    a = x.double()
    b = a.unflatten(-1, (-1, 16))
    fine = torch.isfinite(b)
    mag = torch.where(fine, b.abs(), 0.0)
    m, e = torch.frexp(mag.amax((1, 2, 3)) / 2688.0)
    # (8 significant bits: through fp32, since the GPU's ldexp may be off by a step of its type)
    gs = torch.ldexp(torch.ceil(m * 256), e - 8).clamp(min=2.0 ** -100).float().double()
    g = gs.view(-1, 1, 1)
    bs = _nearest(mag.amax(-1) / (6 * g), E4M3)
    s = (torch.tensor(E4M3, dtype=torch.float64, device=x.device)[bs] * g).unsqueeze(-1)
    code = _nearest(torch.where(s > 0, mag / s, 0.0), E2M1) + 8 * torch.signbit(b)
    bad = ~fine.all(-1)
    code = torch.where(bad.unsqueeze(-1), 0, code).flatten(-2)
    return ((code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), torch.where(bad, 0x7f, bs).to(torch.uint8), gs.float())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2000, 64, 544), (5000, 2, 64), (3, 8192, 2080)])
def test_many_matrices_each_by_its_own_maximum(cuda_lib, shape, dtype):
    """More chunks than the GPU holds at once, the last of a matrix short of a
    whole one: each matrix is coded by its own scale, compared in full."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp2(8 * torch.randn((shape[0], 1, 1), generator=g, device=DEV))
    x = x.to(dtype)
    x[1] = 0.0
    x[2, 1, 5] = float("nan")
    x[-1, -1, -1] *= 1000.0  # the maximum in the last block
    st = cuda_lib.new_status()
    q, bs, gs = cuda_lib.quantize_nvfp4(x, status=st)
    assert int(st.item()) == cuda_lib.MOE_DEV_NONFINITE
    step = max(1, (1 << 26) // (shape[1] * shape[2]))
    for i in range(0, shape[0], step):
        dq, dbs, dgs = _definition(x[i:i + step])
        assert torch.equal(gs[i:i + step], dgs) and torch.equal(bs[i:i + step], dbs) and torch.equal(q[i:i + step], dq), i
