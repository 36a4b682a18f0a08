"""Long sums of the NVFP4 product, which keeps one accumulator: what its
truncating additions (of 64 terms each) take stays within what moe.h states."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(api, counts, N, K, one_sign):
    g = torch.Generator(device=DEV)
    g.manual_seed(K)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)

    def draw(*s):
        t = torch.rand(s, generator=g, device=DEV) + 0.5 if one_sign else torch.randn(s, generator=g, device=DEV)
        # block scales of many bits: the products' sums then have as many
        return t * torch.exp(2 * torch.randn((*s[:-1], K // 16), generator=g, device=DEV)).repeat_interleave(16, -1)

    xq, wq = api.quantize_nvfp4(draw(sum(counts), K)), api.quantize_nvfp4(draw(len(counts), N, K))
    xv, wv = api.dequantize_nvfp4(*xq).double(), api.dequantize_nvfp4(*wq).double()
    segs = list(zip(range(len(counts)), off[:-1].tolist(), off[1:].tolist()))
    y = torch.cat([xv[a:b] @ wv[e].T for e, a, b in segs])
    m = torch.cat([xv[a:b].abs() @ wv[e].abs().T for e, a, b in segs])
    return off, xq, wq, y, m


@pytest.mark.parametrize("one_sign", [True, False])
@pytest.mark.parametrize("counts,N", [([300], 1024), ([60], 1024)])
def test_long_sums_lose_no_more_than_stated(cuda_lib, counts, N, one_sign):
    """K = 16384: 256 additions that truncate, each by less than a step 2^-23
    of a running sum that is half of the result on average: 2^-16 of the
    result, of one sign or in the 2-norm."""
    off, xq, wq, y, _ = _case(cuda_lib, counts, N, 16384, one_sign)
    got = cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off).double()
    assert float((got - y).norm() / y.norm()) <= 2.0 ** -16
    if one_sign:
        assert abs(float((got / y - 1).mean())) <= 2.0 ** -16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [4096, 4128, 8192, 12320])
@pytest.mark.parametrize("counts,N", [([300, 0, 257], 520), ([5, 0, 40, 33], 136), ([160], 264)])
def test_long_sums_that_end_inside_a_stage(cuda_lib, counts, N, K, dtype):
    """Whole stages, and a last one of a few elements.  (K + 1) 2^-23 of the
    magnitudes' sum, two roundings 2^-24, half a step 2^-8 of a bf16 result."""
    off, xq, wq, y, m = _case(cuda_lib, counts, N, K, False)
    R = sum(counts)
    out = torch.full((R + 3, N), -7.0, dtype=dtype, device=DEV)
    xq = tuple(torch.cat([t, t[:3]]) for t in xq)  # rows behind the last segment
    st = cuda_lib.new_status()
    cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out=out, status=st)
    tol = ((K + 1) * 2.0 ** -23 + 2 * 2.0 ** -24) * m
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (y.abs() + tol)
    assert bool(((out[:R].double() - y).abs() <= tol).all())
    assert bool((out[R:] == -7).all()) and int(st.item()) == 0
    assert torch.equal(out, cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out=out.clone()))
