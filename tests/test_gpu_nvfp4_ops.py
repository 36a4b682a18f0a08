"""NVFP4 quantisation, its inverse and the grouped NVFP4 product.

The quantisation is defined on exact arithmetic, so its codes, scales and
values are compared for equality with a 64-bit evaluation of the definition.
The product sums K exact products in fp32, in any order and with additions
that may truncate: (K + 1) 2^-23 of the magnitudes' sum, two roundings by the
scales (2^-24 each) and, in bf16, half a step 2^-8 of the result."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda"
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def _nearest(a, table):
    """Index of the nearest entry of an ascending table, ties to the even index."""
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def _definition(x):
    """[rows, cols] -> (q, bs, gs) of one group, from the definition in 64 bits."""
    a = x.astype(np.float64)
    b = a.reshape(a.shape[0], -1, 16)
    fine = np.isfinite(b)
    mag = np.where(fine, np.abs(b), 0.0)
    top = mag.max() if mag.size else 0.0
    gs = 0.0
    if top > 0:
        m, e = math.frexp(top / 2688.0)
        gs = math.ldexp(math.ceil(m * 256), e - 8)
    gs = max(gs, 2.0 ** -100)
    gs = min(gs, float(np.array([0x79c30000], np.uint32).view(np.float32)[0]))
    bs = _nearest(mag.max(-1) / (6 * gs), E4M3)
    s = E4M3[bs][..., None] * gs
    with np.errstate(divide="ignore", invalid="ignore"):
        code = _nearest(np.where(s > 0, mag / s, 0.0), E2M1) | (np.signbit(b) * 8)
    bad = ~fine.all(-1)
    code[bad] = 0
    bs = np.where(bad, 0x7f, bs)
    code = code.reshape(a.shape).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), bs.astype(np.uint8), np.float32(gs)


def _check_quant(api, x, status=0):
    st = api.new_status()
    q, bs, gs = api.quantize_nvfp4(x, status=st)
    assert int(st.item()) == status
    xn = x.float().cpu().numpy()
    xn = xn[:, None] if x.dim() == 2 else xn
    for i in range(x.shape[0]):
        dq, dbs, dgs = _definition(xn[i])
        assert float(gs[i]) == float(dgs), i
        np.testing.assert_array_equal(bs[i].cpu().numpy().reshape(dbs.shape), dbs)
        np.testing.assert_array_equal(q[i].cpu().numpy().reshape(dq.shape), dq)
    return q, bs, gs


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (5, 512), (7, 544), (2, 2048), (3, 4128), (2, 16384), (1, 1, 32),
                                   (3, 5, 96), (2, 300, 768), (65, 2, 64)])
def test_codes_and_scales_are_the_definition_s(cuda_lib, shape, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(shape))
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(2 * torch.randn((*shape[:-1], 1), generator=g, device=DEV))
    _check_quant(cuda_lib, x.to(dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_zeros_and_the_range_s_ends(cuda_lib, dtype):
    # block maxima 6 * 2^k make the scales powers of two: every quarter step is a tie or a code
    x = torch.zeros((9, 8, 64), device=DEV)
    steps = torch.arange(-24, 24, device=DEV) / 4
    x[0, :, :48] = steps
    x[0, 0, 63] = 2688.0           # gs = 1
    x[0, 1:, 16 * 3] = 6.0
    x[1] = 0.0
    x[2, 0, 0] = -0.0
    x[2, 3, 5] = 1e-38
    x[3] = 3.3e38
    x[3, 1] = -3.3e38
    x[4, 0, 0] = 1.0
    x[4, 1] = 2.0 ** -30           # block scale rounds to zero
    x[4, 2] = 6 * 2.0 ** -9 / 2688.0
    x[5] = torch.randint(-7, 8, (8, 64), device=DEV).float()
    x[6] = torch.randint(-100, 101, (8, 64), device=DEV).float() / 16
    x[7] = 2.0 ** -140
    x[8] = torch.linspace(-1, 1, 512, device=DEV).view(8, 64)
    _check_quant(cuda_lib, x.to(dtype))
    _check_quant(cuda_lib, x.to(dtype).view(72, 64))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_blocks_that_are_not_finite_decode_to_nan_and_leave_the_others(cuda_lib, dtype, bad):
    x = torch.randn((4, 3, 96), device=DEV).to(dtype)
    x[1, 2, 17] = bad
    for t in (x, x.view(12, 96)):
        q, bs, gs = _check_quant(cuda_lib, t, cuda_lib.MOE_DEV_NONFINITE)
        v = cuda_lib.dequantize_nvfp4(q, bs, gs).view(4, 3, 6, 16)
        want = torch.zeros((4, 3, 6), dtype=torch.bool, device=DEV)
        want[1, 2, 1] = True
        assert torch.equal(torch.isnan(v).all(-1), want) and torch.equal(torch.isnan(v).any(-1), want)


@pytest.mark.parametrize("shape", [(5, 96), (3, 7, 160), (2, 33, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_of_any_codes_and_scales(cuda_lib, shape, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    *lead, cols = shape
    q = torch.randint(0, 256, (*lead, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    bs = torch.randint(0, 127, (*lead, cols // 16), generator=g, device=DEV, dtype=torch.uint8)
    gs = torch.randn(shape[0], generator=g, device=DEV).abs()
    got = cuda_lib.dequantize_nvfp4(q, bs, gs, out_dtype=dtype)
    for i in range(shape[0]):
        want = torch.from_numpy(oracle.dequant_nvfp4(q[i].view(-1, cols // 2).cpu().numpy(), bs[i].view(-1, cols // 16).cpu().numpy(),
                                                     float(gs[i])))
        assert torch.equal(got[i].view(-1, cols).cpu(), want.to(dtype))


def _product_case(counts, N, K, seed=0, trail=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    R = sum(counts) + trail
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
    x = torch.randn((R, K), generator=g, device=DEV) * torch.exp(torch.randn((R, 1), generator=g, device=DEV))
    w = torch.randn((len(counts), N, K), generator=g, device=DEV) * 0.05
    return off, x, w


def _check_product(api, off, xq, wq, y, rows=None):
    x, w = api.dequantize_nvfp4(*xq).double(), api.dequantize_nvfp4(*wq).double()
    K = x.shape[1]
    for e in range(w.shape[0]):
        s = slice(int(off[e]), int(off[e + 1]))
        if rows is not None and not (rows.start <= s.start and s.stop <= rows.stop):
            continue
        ref, m = x[s] @ w[e].T, x[s].abs() @ w[e].abs().T
        tol = ((K + 1) * 2.0 ** -23 + 2 * 2.0 ** -24) * m
        if y.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        d = (y[s].double() - ref).abs()
        assert bool((d <= tol).all()), (e, float((d / tol.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 32),
    ([0, 3, 0, 1], 128, 256),
    ([2, 0, 1, 1, 0], 1536, 2048),
    ([5, 0, 40, 33], 136, 96),       # rows of scales that are not whole words
    ([1, 64, 0, 130], 264, 448),     # ... whole words
    ([300, 0, 257], 520, 1280),
    ([7] * 60, 64, 768),
])
def test_product_matches_64_bits(cuda_lib, counts, N, K, dtype):
    off, x, w = _product_case(counts, N, K)
    xq, wq = cuda_lib.quantize_nvfp4(x), cuda_lib.quantize_nvfp4(w)
    st = cuda_lib.new_status()
    y = cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out_dtype=dtype, status=st)
    _check_product(cuda_lib, off, xq, wq, y)
    assert int(st.item()) == 0


@pytest.mark.parametrize("counts", [[2, 0, 1], [40, 0, 61], [300, 0, 200]])
def test_product_edges(cuda_lib, counts):
    """Rows behind the last segment stay; NaN blocks stay in their row and
    expert; the same bits again, captured and on another stream."""
    off, x, w = _product_case(counts, 72, 160, trail=4)
    n = sum(counts)
    x[int(off[-2]):, 3] = float("nan")
    w[1, 5, 7] = float("inf")
    xq, wq = cuda_lib.quantize_nvfp4(x), cuda_lib.quantize_nvfp4(w)
    out = torch.full((n + 4, 72), -7.0, device=DEV)
    cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out=out)
    _check_product(cuda_lib, off, xq, wq, out, slice(0, int(off[-2])))
    assert bool(torch.isnan(out[int(off[-2]):n]).all()) and bool((out[n:] == -7).all())
    first = out.nan_to_num(1.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, out.nan_to_num(1.5))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off, out=out)
    out.fill_(-7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out.nan_to_num(1.5))
    bad = off.clone()
    bad[1] = n + 5
    st = cuda_lib.new_status()
    cuda_lib.grouped_gemm_nvfp4(*xq, *wq, bad, out=out, status=st)
    assert int(st.item()) == cuda_lib.MOE_DEV_BAD_OFFSETS
    out.fill_(-7.0)
    cuda_lib.grouped_gemm_nvfp4(*xq, *wq, torch.full_like(off, 2), out=out)  # no segment holds a row
    assert bool((out == -7).all())
    assert cuda_lib.grouped_gemm_nvfp4(*(t[:0] for t in xq), *wq, torch.zeros_like(off)).shape == (0, 72)


def test_quantising_again_captured_and_on_another_stream(cuda_lib):
    x = torch.randn((5, 40, 96), device=DEV)
    first = cuda_lib.quantize_nvfp4(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = cuda_lib.quantize_nvfp4(x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    out = tuple(torch.empty_like(t) for t in first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda_lib.quantize_nvfp4(x, out=out)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, out):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_quantised_weights_run_in_the_stack_and_in_the_product(cuda_lib):
    """Weights quantised here drive moe_stack_forward_nvfp4 as the recipe's
    do, and the same layer from quantise + grouped products is within what
    4-bit activations cost of it."""
    from moe_decode_layer_gemv_gb300 import synth
    w = synth.Workload("nvfp4", B=48, H=256, I=128, E=8, top_k=2, sigma_router=256 ** -0.5, sigma_expert=0.05)
    lw = synth.make_layer(w, 0, seed=2, device=DEV)
    for n in ("gate_up", "down"):
        lw[n + "_q4"], lw[n + "_bs"], lw[n + "_gs"] = cuda_lib.quantize_nvfp4(lw[n])
    x = synth.make_x(w, 0, seed=2, device=DEV)
    st = cuda_lib.new_status()
    ids = torch.empty((1, w.B, w.top_k), dtype=torch.int32, device=DEV)
    y = cuda_lib.stack_forward_nvfp4_(x.clone(), cuda_lib.StackWeightsNVFP4([lw]), w.top_k, ids_out=ids, status=st) - x
    assert int(st.item()) == 0
    dq = {n: cuda_lib.dequantize_nvfp4(lw[n + "_q4"], lw[n + "_bs"], lw[n + "_gs"]) for n in ("gate_up", "down")}
    _, rw, _ = cuda_lib.route(x, lw["w_router"], w.top_k)
    off, ridx, _, _ = cuda_lib.group_by_expert(ids[0], w.E)
    ridx = ridx.long()

    def layer(gemm):
        gu = gemm(x[ridx // w.top_k].contiguous(), "gate_up")
        h = (torch.nn.functional.silu(gu[:, :w.I]) * gu[:, w.I:]).contiguous()
        o = gemm(h, "down") * rw.flatten()[ridx].unsqueeze(1)
        return torch.zeros_like(x).index_add_(0, ridx // w.top_k, o)

    def exact(a, n):
        return torch.cat([a[int(off[e]):int(off[e + 1])].double() @ dq[n][e].double().T for e in range(w.E)]).float()

    def product(a, n):
        return cuda_lib.grouped_gemm_nvfp4(*cuda_lib.quantize_nvfp4(a), lw[n + "_q4"], lw[n + "_bs"], lw[n + "_gs"], off)

    want = layer(exact)
    assert float((y - want).abs().max()) <= 2e-3 * float(want.abs().max())
    # a code is off by at most a quarter of its magnitude (half a step of 0.5
    # at 1.0 is the coarsest); two quantised operands in a row stay below a half
    assert float((layer(product) - want).norm() / want.norm()) <= 0.5


def test_quantisation_past_32_bits(cuda_lib):
    """More than 2^31 elements: the last matrix, and the last row, against the definition."""
    for shape in ((34, 8192, 8192), (140000, 16384)):
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        x.fill_(0.5)
        g = torch.Generator(device=DEV)
        g.manual_seed(1)
        last = x[-1:].reshape(-1, shape[-1])[:8]
        last.copy_(torch.randn(last.shape, generator=g, device=DEV) * 3)
        q, bs, gs = cuda_lib.quantize_nvfp4(x)
        dq, dbs, dgs = _definition(last.float().cpu().numpy())
        assert float(gs[-1]) == float(dgs)
        np.testing.assert_array_equal(q[-1:].reshape(-1, shape[-1] // 2)[:8].cpu().numpy(), dq)
        np.testing.assert_array_equal(bs[-1:].reshape(-1, shape[-1] // 16)[:8].cpu().numpy(), dbs)
        v = cuda_lib.dequantize_nvfp4(q, bs, gs, out_dtype=torch.bfloat16)
        want = oracle.dequant_nvfp4(dq, dbs, float(dgs))
        assert torch.equal(v[-1:].reshape(-1, shape[-1])[:8].cpu(), torch.from_numpy(want).to(torch.bfloat16))
        del x, q, bs, gs, v
        torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [3, 60, 400])
def test_product_of_the_largest_matrices(cuda_lib, rows):
    off, x, w = _product_case([rows], 2 * cuda_lib.MAX_DIM, cuda_lib.MAX_DIM)
    xq, wq = cuda_lib.quantize_nvfp4(x), cuda_lib.quantize_nvfp4(w)
    del x, w
    y = cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off)
    _check_product(cuda_lib, off, xq, wq, y)
    del y, xq, wq
    torch.cuda.empty_cache()
