"""The grouped products (moe_grouped_gemm, _dx, _dw) against plain loops over
the segments in 64 bits.

Tolerance: a sum of n exact products in fp32, in any order and with additions
that may truncate (one step, 2^-23, of the running sum of magnitudes each),
is within (n + 1) 2^-23 sum |a||b| of the exact value; a result rounded to
bf16 is off by at most half a step more, 2^-8 of its magnitude."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(counts, N, K, seed=0, lead=0, trail=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    R = lead + sum(counts) + trail
    off = lead + np.concatenate([[0], np.cumsum(counts)])
    r = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    return (torch.from_numpy(off.astype(np.int32)).to(DEV), r(R, K), (r(len(counts), N, K) * 0.05).to(torch.bfloat16),
            r(R, N))


def _reference(op, off, x, w, dy):
    """-> (values, magnitude sums, terms of a sum) in 64 bits; None for rows of no segment."""
    off = off.tolist()
    x, w, dy = (t.double() for t in (x, w, dy))
    E, N, K = w.shape
    shape = {"fwd": (x.shape[0], N), "dx": (x.shape[0], K), "dw": (E, N, K)}[op]
    y, m = torch.zeros(shape, dtype=torch.float64, device=DEV), torch.zeros(shape, dtype=torch.float64, device=DEV)
    terms = {"fwd": K, "dx": N, "dw": max(b - a for a, b in zip(off, off[1:]))}[op]
    for e in range(E):
        s = slice(off[e], off[e + 1])
        if op == "fwd":
            y[s], m[s] = x[s] @ w[e].T, x[s].abs() @ w[e].abs().T
        elif op == "dx":
            y[s], m[s] = dy[s] @ w[e], dy[s].abs() @ w[e].abs()
        else:
            y[e], m[e] = dy[s].T @ x[s], dy[s].abs().T @ x[s].abs()
    return y, m, terms


def _call(api, op, off, x, w, dy, **kw):
    if op == "fwd":
        return api.grouped_gemm(x, w, off, **kw)
    if op == "dx":
        return api.grouped_gemm_dx(dy, w, off, **kw)
    return api.grouped_gemm_dw(dy, x, off, **kw)


def _check(got, ref, dtype, rows=slice(None)):
    y, m, terms = ref
    tol = (terms + 1) * 2.0 ** -23 * m[rows]
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (y[rows].abs() + tol)
    d = (got[rows].double() - y[rows]).abs()
    assert bool((d <= tol).all()), float((d / tol.clamp(min=1e-300)).max())


# few rows (the row-at-a-time kernel), single tiles, several tiles with ragged
# ends, and enough rows a segment for the paired tiles
SHAPES = [
    ([1], 8, 8),
    ([0, 2, 0, 0, 1, 0], 1536, 2048),
    ([5, 0, 9], 40, 2056),
    ([1, 0, 40, 31, 0, 130], 264, 200),
    ([33] * 40, 136, 72),
    ([257, 0, 3, 190], 520, 264),
    ([700], 256, 512),
    ([300, 129, 513, 1], 392, 1000),
    ([0, 640, 129, 0, 500], 768, 136),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_matches_64_bit_loops(cuda_lib, op, counts, N, K, dtype):
    off, x, w, dy = _case(counts, N, K)
    st = cuda_lib.new_status()
    got = _call(cuda_lib, op, off, x, w, dy, out_dtype=dtype, status=st)
    assert got.dtype == dtype
    _check(got, _reference(op, off, x, w, dy), dtype)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("op,counts,N,K", [
    ("fwd", [3, 0, 200], 136, 4104), ("fwd", [300, 260], 264, 4104),   # several accumulators a sum
    ("dx", [70, 5], 4104, 136), ("dx", [300, 260], 4104, 264),
    ("dw", [5000], 264, 200), ("dw", [3000, 0, 2100], 136, 72),        # ... and segments cut into parts
    ("dw", [12345, 1, 0, 4000], 64, 520), ("dw", [700, 33000], 72, 72),
])
def test_long_sums_stay_close(cuda_lib, op, counts, N, K, dtype):
    """fp32 results of long contractions: parts of 1024 terms in the tensor
    cores, whose additions may truncate (2^-23 of the part's magnitudes each
    addition of 16 terms, 64 of them: 2^-17; the terms' own sum adds as much
    at most), added with rounding to nearest (2^-24 of the sum's magnitudes
    each).  Errors of a random sign's sum stay far below: what is held here is
    2^-17 of the result's 2-norm, where one accumulator for 33000 terms is off by 2e-5."""
    off, x, w, dy = _case(counts, N, K)
    got = _call(cuda_lib, op, off, x, w, dy, out_dtype=dtype)
    ref = _reference(op, off, x, w, dy)
    _check(got, ref, dtype)
    if dtype == torch.float32:
        assert float((got.double() - ref[0]).norm() / ref[0].norm()) <= 2.0 ** -17


@pytest.mark.parametrize("counts", [[2, 0, 3], [20, 0, 43, 1], [200, 0, 300]])
@pytest.mark.parametrize("op", ["fwd", "dx"])
def test_rows_of_no_segment_are_left_as_they_were(cuda_lib, op, counts):
    off, x, w, dy = _case(counts, 72, 136, lead=3, trail=5)
    ref = _reference(op, off, x, w, dy)
    out = torch.full(ref[0].shape, -7.0, device=DEV)
    _call(cuda_lib, op, off, x, w, dy, out=out)
    _check(out, ref, torch.float32, slice(3, 3 + sum(counts)))
    assert bool((out[:3] == -7).all()) and bool((out[3 + sum(counts):] == -7).all())


@pytest.mark.parametrize("counts", [[2, 0, 1], [17, 0, 21, 30], [150, 0, 290, 141]])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row_and_expert(cuda_lib, op, counts, bad):
    """Rows of the last segment are not finite, and so is the empty expert's
    matrix: the other segments' results are those of finite inputs, although
    their tiles reach into those rows."""
    off, x, w, dy = _case(counts, 72, 136)
    first = int(off[-2])
    ref = _reference(op, off, x, w, dy)
    x[first:], dy[first:], w[1] = bad, bad, bad
    got = _call(cuda_lib, op, off, x, w, dy)
    keep = slice(0, len(counts) - 1) if op == "dw" else slice(0, first)
    _check(got, ref, torch.float32, keep)
    assert not bool(torch.isfinite(got[-1]).any())


def test_experts_without_rows_get_zero_gradients(cuda_lib):
    off, x, w, dy = _case([0, 5, 0], 72, 136)
    out = torch.full((3, 72, 136), 9.0, dtype=torch.bfloat16, device=DEV)
    cuda_lib.grouped_gemm_dw(dy, x, off, out=out)
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
    # no rows at all: zeros, and empty outputs of the other two
    none = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert bool((cuda_lib.grouped_gemm_dw(dy[:0], x[:0], none) == 0).all())
    assert cuda_lib.grouped_gemm(x[:0], w, none).shape == (0, 72)
    assert cuda_lib.grouped_gemm_dx(dy[:0], w, none).shape == (0, 136)
    # rows, but no segment that holds them
    out.fill_(9.0)
    cuda_lib.grouped_gemm_dw(dy, x, none, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("rows", [6, 60, 600])
@pytest.mark.parametrize("op", ["fwd", "dx"])
def test_rows_without_any_segment(cuda_lib, op, rows):
    _, x, w, dy = _case([rows, 0, 0], 40, 72)
    out = torch.full((rows, 40 if op == "fwd" else 72), -7.0, device=DEV)
    st = cuda_lib.new_status()
    _call(cuda_lib, op, torch.full((4,), 5, dtype=torch.int32, device=DEV), x, w, dy, out=out, status=st)
    assert bool((out == -7).all()) and int(st.item()) == 0


def test_two_streams_at_once(cuda_lib):
    """Calls of every kind in flight together: none shares state with another."""
    cases = [_case(c, 264, 200, seed=i) for i, c in enumerate(([3, 1], [30, 50, 0, 11], [400, 0, 250], [9000]))]
    want = [[_call(cuda_lib, op, *c) for op in ("fwd", "dx", "dw")] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cases, streams)):
            got[i] = [_call(cuda_lib, op, *c, stream=s) for op in ("fwd", "dx", "dw")]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,k,E", [(4, 2, 40), (100, 4, 24), (700, 2, 6)])
def test_inputs_written_by_the_call_before(cuda_lib, B, k, E):
    """Each call's inputs are written right before it on the stream (launches
    overlap the end of the kernel ahead): rows, weights and the grouping
    change every time, in the same buffers."""
    N, K, g = 72, 136, torch.Generator(device=DEV)
    g.manual_seed(0)
    x = torch.empty((B * k, K), dtype=torch.bfloat16, device=DEV)
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    seen = []
    for _ in range(20):
        ids = torch.rand((B, E), generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
        nx, nw = torch.randn_like(x), torch.randn_like(w)
        x.copy_(nx), w.copy_(nw)
        off.copy_(cuda_lib.group_by_expert(ids, E)[0])
        y = cuda_lib.grouped_gemm(x, w, off)
        dx = cuda_lib.grouped_gemm_dx(y.to(torch.bfloat16), w, off)
        q = cuda_lib.grouped_gemm_nvfp4(*cuda_lib.quantize_nvfp4(torch.nn.functional.pad(x, (0, 24))),
                                        *cuda_lib.quantize_nvfp4(torch.nn.functional.pad(w, (0, 24))), off)
        seen.append((nx, nw, off.clone(), y, dx, q))
    torch.cuda.synchronize()
    for nx, nw, o, y, dx, q in seen:
        x.copy_(nx), w.copy_(nw), off.copy_(o)
        torch.cuda.synchronize()
        assert torch.equal(y, cuda_lib.grouped_gemm(x, w, off))
        yb = y.to(torch.bfloat16)
        torch.cuda.synchronize()
        assert torch.equal(dx, cuda_lib.grouped_gemm_dx(yb, w, off))
        xq = cuda_lib.quantize_nvfp4(torch.nn.functional.pad(x, (0, 24)))
        wq = cuda_lib.quantize_nvfp4(torch.nn.functional.pad(w, (0, 24)))
        torch.cuda.synchronize()
        assert torch.equal(q, cuda_lib.grouped_gemm_nvfp4(*xq, *wq, off))


@pytest.mark.parametrize("rows", [6, 60, 600])
@pytest.mark.parametrize("offsets", [[0, 4, 2, 6], [-1, 2, 3, 6], [0, 2, 3, 7], [0, 2 ** 31 - 1, 2, 6]])
@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_bad_offsets_leave_their_segment_out(cuda_lib, op, offsets, rows):
    scale = rows // 6
    off = torch.tensor([o if abs(o) > 9 else o * scale for o in offsets], dtype=torch.int32, device=DEV)
    _, x, w, dy = _case([rows, 0, 0], 40, 72)
    st = cuda_lib.new_status()
    _call(cuda_lib, op, off, x, w, dy, status=st)
    assert int(st.item()) == cuda_lib.MOE_DEV_BAD_OFFSETS


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("counts", [[3, 1], [30, 50, 0, 11], [400, 0, 250]])
def test_bit_for_bit_again_captured_and_on_another_stream(cuda_lib, op, counts):
    off, x, w, dy = _case(counts, 264, 200)
    first = _call(cuda_lib, op, off, x, w, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = _call(cuda_lib, op, off, x, w, dy, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, other)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(cuda_lib, op, off, x, w, dy, out=out)
    out.fill_(-1)
    # other segment sizes at replay: the launch does not depend on them
    off2 = off.clone()
    off2[1:-1] = off[1:-1] // 2
    keep = off.clone()
    off.copy_(off2)
    g.replay()
    torch.cuda.synchronize()
    _check(out, _reference(op, off, x, w, dy), torch.float32)
    off.copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)


def test_gradients_against_differences(cuda_lib):
    """d/dt of the loss sum(y * dy) along directions of x and w, by central
    differences of the product itself, against dx and dw.  The product is
    linear in each, so the difference quotient is the derivative and what is
    left is fp32 rounding of y (bounded like the sums above) and of the
    results: 64 times 2^-23 of the magnitudes' sum covers both at K, N, rows
    below 200."""
    off, x, w, dy = _case([3, 0, 40, 160], 136, 72)
    vx = torch.randint(-1, 2, x.shape, device=DEV).to(torch.bfloat16)
    vw = torch.randint(-1, 2, w.shape, device=DEV).to(torch.bfloat16)
    loss = lambda y: (y.double() * dy.double()).sum()  # noqa: E731
    dx = cuda_lib.grouped_gemm_dx(dy, w, off)
    dw = cuda_lib.grouped_gemm_dw(dy, x, off)
    up, down = (x.float() + vx.float()).to(torch.bfloat16), (x.float() - vx.float()).to(torch.bfloat16)
    moved = (up.double() - down.double()) / 2  # the step as rounded to bf16
    num = (loss(cuda_lib.grouped_gemm(up, w, off)) - loss(cuda_lib.grouped_gemm(down, w, off))) / 2
    _, m, terms = _reference("fwd", off, up.abs() + down.abs(), w, dy)
    tol = 64 * terms * 2.0 ** -23 * float((m * dy.double().abs()).sum())
    assert abs(float(num - (dx.double() * moved).sum())) <= tol
    up, down = (w.float() + vw.float()).to(torch.bfloat16), (w.float() - vw.float()).to(torch.bfloat16)
    moved = (up.double() - down.double()) / 2
    num = (loss(cuda_lib.grouped_gemm(x, up, off)) - loss(cuda_lib.grouped_gemm(x, down, off))) / 2
    _, m, terms = _reference("fwd", off, x, up.abs() + down.abs(), dy)
    tol = 64 * terms * 2.0 ** -23 * float((m * dy.double().abs()).sum())
    assert abs(float(num - (dw.double() * moved).sum())) <= tol


def test_a_layer_of_grouped_products_matches_the_expert_pass(cuda_lib):
    """route -> group -> gather -> gate/up -> SiLU*up -> down -> combine with
    the grouped products, against moe_expert_forward on the same routing, and
    its gradients against autograd through the same formulas in 64 bits."""
    from moe_decode_layer_gemv_gb300 import synth
    w = synth.Workload("grouped", B=96, H=256, I=128, E=12, top_k=3, sigma_router=256 ** -0.5, sigma_expert=0.05)
    lw = synth.make_layer(w, 0, seed=1, device=DEV)
    x = synth.make_x(w, 0, seed=1, device=DEV).to(torch.bfloat16)
    ids, rw, _ = cuda_lib.route(x, lw["w_router"], w.top_k)
    grouping = cuda_lib.group_by_expert(ids, w.E)
    want = cuda_lib.expert_forward(x, lw["gate_up"], lw["down"], ids, rw, grouping)
    off, ridx = grouping[0], grouping[1].long()
    xs = x[ridx // w.top_k]
    gu = cuda_lib.grouped_gemm(xs, lw["gate_up"], off)
    h = (torch.nn.functional.silu(gu[:, :w.I]) * gu[:, w.I:])
    hb = h.to(torch.bfloat16)
    o = cuda_lib.grouped_gemm(hb, lw["down"], off)
    y = torch.zeros_like(want).index_add_(0, ridx // w.top_k, o * rw.flatten()[ridx].unsqueeze(1))
    # h in bf16 (half a step 2^-8 an element) where the layer splits it into two parts
    d, m = lw["down"].double(), torch.zeros_like(want, dtype=torch.float64)
    for e in range(w.E):
        s = slice(int(off[e]), int(off[e + 1]))
        m.index_add_(0, ridx[s] // w.top_k, (h[s].double().abs() @ d[e].abs().T) * rw.flatten()[ridx[s]].double().unsqueeze(1))
    assert bool(((y - want).double().abs() <= (2.0 ** -8 + 2.0 ** -12) * m).all())
    # the training step: gradients of sum(y * g)
    g = torch.randn(want.shape, device=DEV)
    do = (g[ridx // w.top_k] * rw.flatten()[ridx].unsqueeze(1)).to(torch.bfloat16)
    dh = cuda_lib.grouped_gemm_dx(do, lw["down"], off)
    d_down = cuda_lib.grouped_gemm_dw(do, hb, off)
    gate, up = gu[:, :w.I], gu[:, w.I:]
    sig = torch.sigmoid(gate)
    dgu = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1).to(torch.bfloat16)
    d_gate_up = cuda_lib.grouped_gemm_dw(dgu, xs, off)
    dxs = cuda_lib.grouped_gemm_dx(dgu, lw["gate_up"], off)
    X, G, D = (t.double().requires_grad_() for t in (xs, lw["gate_up"], lw["down"]))
    loss = 0.0
    for e in range(w.E):
        s = slice(int(off[e]), int(off[e + 1]))
        a = X[s] @ G[e].T
        loss = loss + ((torch.nn.functional.silu(a[:, :w.I]) * a[:, w.I:]) @ D[e].T * do[s].double()).sum()
    loss.backward()
    # bf16 steps on the way (h; dgu): half a step each, 2^-8, relative to the
    # largest magnitudes that enter a sum, whose errors are independent
    for got, ref in ((d_down, D.grad), (d_gate_up, G.grad), (dxs, X.grad)):
        assert float((got.double() - ref).norm() / ref.norm()) <= 2 * 2.0 ** -8


def _sampled(cuda_lib, op, off, x, w, dy, rows):
    """The result of a large case at some of its segments (dw) or rows."""
    got = _call(cuda_lib, op, off, x, w, dy, out_dtype=torch.bfloat16)
    o = off.tolist()
    for at in rows:
        e = at if op == "dw" else next(i for i in range(len(o) - 1) if o[i] <= at < o[i + 1])
        if op == "dw":
            s = slice(o[e], o[e + 1])
            terms, y, m = o[e + 1] - o[e], dy[s].double().T @ x[s].double(), dy[s].double().abs().T @ x[s].double().abs()
        elif op == "fwd":
            terms, y, m = x.shape[1], w[e].double() @ x[at].double(), w[e].double().abs() @ x[at].double().abs()
        else:
            terms, y, m = dy.shape[1], dy[at].double() @ w[e].double(), dy[at].double().abs() @ w[e].double().abs()
        tol = (terms + 1) * 2.0 ** -23 * m
        assert bool(((got[at].double() - y).abs() <= tol + 2.0 ** -8 * (y.abs() + tol)).all()), at
    return got


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_offsets_past_32_bits(cuda_lib, op):
    """More than 2^31 elements in the row tensor, or in the gradient of the weights."""
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    if op == "dw":
        E, R, N, K = 40, 400, 8192, 8192
        off = torch.arange(0, R + 1, R // E, dtype=torch.int32, device=DEV)
        _sampled(cuda_lib, op, off, r(R, K), r(1, 8, 8), r(R, N), (0, 33, 39))
    else:
        R, N, K = 1_100_000, 2048, 64
        off = torch.tensor([0, 1_000_000, 1_000_000, R], dtype=torch.int32, device=DEV)
        if op == "dx":
            N, K = K, N
        _sampled(cuda_lib, op, off, r(R, K) if op == "fwd" else r(1, 8), r(3, N, K), r(R, N) if op == "dx" else r(1, 8),
                 (0, 999_999, 1_000_000, 1_060_000, R - 1))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
@pytest.mark.parametrize("counts", [[3], [40], [300]])
def test_the_largest_matrices(cuda_lib, op, counts):
    off, x, w, dy = _case(counts, 2 * cuda_lib.MAX_DIM, cuda_lib.MAX_DIM)
    _sampled(cuda_lib, op, off, x, w, dy, (0,) if op == "dw" else (0, counts[0] - 1))
    torch.cuda.empty_cache()


@pytest.mark.parametrize("op", ["fwd", "dx", "dw"])
def test_the_most_rows_and_segments(cuda_lib, op):
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    R, N, K, E = cuda_lib.MAX_ROWS, 72, 40, cuda_lib.MAX_E
    off = (torch.arange(E + 1, dtype=torch.int64) * 16363).clamp(max=R).to(torch.int32)
    off[-1] = R
    _sampled(cuda_lib, op, off.to(DEV), r(R, K), r(E, N, K), r(R, N), (0, 7, 255) if op == "dw" else (0, 16362, 16363, R - 1))
