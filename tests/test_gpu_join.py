"""What joins a block to the residual stream (moe_combine_norm) and its
gradients, against the formulas in 64 bits.

Tolerances, token by token, in 2-norms.  A sum of H products in fp32 is taken
by at most 64 columns a thread and a tree of ten additions: it is within
2^-17 |a||b| (Cauchy-Schwarz; 74 steps of 2^-24), and a norm's factor within
2^-17 of itself.  z is off by e = (k + 1) 2^-24 sum |w||o|, which moves its
direction by p = |e| / max(|z|, sqrt(H eps)).  What follows from that:
  b:   (2^-16 + 2 p) |b|, or |e| without a norm behind the block
  y:   |scale b|'s error + 2^-22 (|x| + |scale b|)
  n:   (2^-16 + 2 |y's error| / max(|y|, sqrt(H eps))) |n|
  d = dx:  q = 2^-16 (|dy| + 2 rms(y) |dn pre|)
  dz:  2 rms(z) |post scale|max q + 4 (2^-16 + p) rms(z) |c|  (without a norm: |scale|max q)
  dw:  |o_j| (dz's + 2^-17 |dz|);   do: |w_j| dz's
(r a - y r^3 mean(a y) is no larger than 2 r |a|).  Column sums add T terms:
the terms' own errors, and 2^-24 T of their magnitudes at most.  A result
rounded to bf16 is off by at most half a step more, 2^-8 of its magnitude."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def _case(T, k, H, x=F32, o=BF16, n=BF16, drop=0.0, post=True, scale=True, pre=True, w=True, pos=True, rows=True, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    c = dict(x=(r(T, H) * torch.exp(r(T, 1))).to(x), dy=(r(T, H) * 0.1).to(x), dn=(r(T, H) * 0.1).to(n) if pre else None,
             pre=1 + 0.1 * r(H) if pre else None, eps=EPS, n_dtype=n, o=None, pos=None, w=None, post=None, scale=1.0)
    if not rows:
        return c
    R = T * k
    c["o"] = r(R, H).to(o)
    if pos:
        p = torch.randperm(R, generator=g, device=DEV).int()
        c["pos"] = torch.where(torch.rand(R, generator=g, device=DEV) < drop, -1, p).view(T, k)
    if w:
        c["w"] = torch.softmax(r(T, k), 1)
    if post:
        c["post"] = 1 + 0.1 * r(H)
    c["scale"] = 0.5 + 0.1 * r(H) if scale else 0.75
    return c


def _d(t):
    return t.double() if torch.is_tensor(t) else t


def _norms(t):
    return t.norm(dim=-1)


def _z(c):
    """z, the rows that went into it [T, k, H] (zeros for none), the weights, z's errors."""
    T, H = c["x"].shape
    if c["o"] is None:
        return (torch.zeros((T, H), dtype=torch.float64, device=DEV),) + (None,) * 3
    o = torch.cat([c["o"].double(), torch.zeros((1, H), dtype=torch.float64, device=DEV)])
    k = c["pos"].shape[1] if c["pos"] is not None else c["w"].shape[1] if c["w"] is not None else o.shape[0] // T
    pos = c["pos"].long() if c["pos"] is not None else torch.arange(T * k, device=DEV).view(T, k)
    rows = o[torch.where(pos < 0, -1, pos)]
    w = _d(c["w"]) if c["w"] is not None else torch.ones((T, k), dtype=torch.float64, device=DEV)
    e = (k + 1) * 2.0 ** -24 * (w.abs().unsqueeze(2) * rows.abs()).sum(1)
    return (w.unsqueeze(2) * rows).sum(1), rows, w, e


def _rms(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _forward(c):
    x, (z, _, _, e) = _d(c["x"]), _z(c)
    e = None if e is None else _norms(e)
    floor = (x.shape[1] * EPS) ** 0.5
    if c["o"] is None:
        y, ey = x, torch.zeros(x.shape[0], device=DEV, dtype=torch.float64)
    else:
        if c["post"] is not None:
            b = z * _rms(z) * _d(c["post"])
            eb = (2.0 ** -16 + 2 * e / _norms(z).clamp(min=floor)) * _norms(b) * 2
        else:
            b, eb = z, e
        s = _d(c["scale"])
        top = s.abs().max() if torch.is_tensor(s) else abs(s)
        y = x + s * b
        ey = top * eb + 2.0 ** -22 * (_norms(x) + _norms(s * b))
    out = [(y, ey)]
    if c["pre"] is not None:
        n = y * _rms(y) * _d(c["pre"])
        out.append((n, (2.0 ** -16 + 4 * ey / _norms(y).clamp(min=floor)) * _norms(n)))
    return out


def _backward(c):
    """-> {name: (value, tolerance)}; rows' tolerances are of their 2-norms, columns' of each value."""
    y, T = _d(c["x"]), c["x"].shape[0]
    floor = (y.shape[1] * EPS) ** 0.5
    z, rows, w, e = _z(c)
    d = _d(c["dy"]) if c["dy"] is not None else torch.zeros_like(y)
    q, out = 2.0 ** -16 * _norms(d), {}
    many = 2.0 ** -24 * T
    if c["pre"] is not None:
        r, dn = _rms(y), _d(c["dn"])
        a = dn * _d(c["pre"])
        out["dpre"] = ((dn * y * r).sum(0), (2.0 ** -16 + many) * (dn * y * r).abs().sum(0))
        d = d + r * a - y * r ** 3 * (a * y).mean(1, keepdim=True)
        q = q + 2.0 ** -15 * r.flatten() * _norms(a)
    out["dx"] = (d, q)
    if rows is None:
        return out
    s = _d(c["scale"])
    top = s.abs().max() if torch.is_tensor(s) else abs(s)
    rz, p = _rms(z), _norms(e) / _norms(z).clamp(min=floor)
    hat = z * rz
    b = hat * _d(c["post"]) if c["post"] is not None else z
    # of one column: z's own error e there (where the rows cancel it is not small beside z), times
    # rms(z) post with a norm behind the block, and what the norm's factor adds in proportion
    if torch.is_tensor(s):
        t = d * b
        if c["post"] is not None:
            eb = (2.0 ** -16 + 4 * p) * b.abs().T + 2 * (rz * e * _d(c["post"]).abs()).T
        else:
            eb = 2.0 ** -22 * b.abs().T + e.T
        out["dscale"] = (t.sum(0), (b.abs().T * q + d.abs().T * eb).sum(1) + many * t.abs().sum(0))
    g = s * d
    if c["post"] is not None:
        t = g * hat
        out["dpost"] = (t.sum(0), (hat.abs().T * q * top + t.abs().T * (2.0 ** -16 + 4 * p) + 2 * (g.abs() * rz * e).T).sum(1) + many * t.abs().sum(0))
        post = _d(c["post"])
        f = g * post
        dz = rz * f - z * rz ** 3 * (f * z).mean(1, keepdim=True)
        ez = rz.flatten() * (2 * post.abs().max() * top * q + 4 * (2.0 ** -16 + p) * _norms(f))
    else:
        dz, ez = g, top * q + 2.0 ** -23 * _norms(g)
    do = torch.full((c["o"].shape[0] + 1, y.shape[1]), -7.0, dtype=torch.float64, device=DEV)
    tol = torch.zeros(c["o"].shape[0] + 1, dtype=torch.float64, device=DEV)
    pos = c["pos"].long() if c["pos"] is not None else torch.arange(w.numel(), device=DEV).view(w.shape)
    pos = torch.where(pos < 0, c["o"].shape[0], pos)
    do[pos] = w.unsqueeze(2) * dz.unsqueeze(1)
    tol[pos] = w.abs() * (ez + 2.0 ** -23 * _norms(dz)).unsqueeze(1)
    out["do"] = (do[:-1], tol[:-1])
    if c["w"] is not None:
        out["dw"] = ((dz.unsqueeze(1) * rows).sum(2), _norms(rows) * (ez + 2.0 ** -17 * _norms(dz)).unsqueeze(1))
    return out


def _near_rows(got, want, tol):
    half = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    off, tol = _norms(got.double() - want), tol + half * (_norms(want) + tol) + 1e-30
    assert bool((off <= tol).all()), float((off / tol).max())


def _near(got, want, tol):
    off, tol = (got.double() - want).abs(), tol + 2.0 ** -24 * want.abs() + 1e-30
    assert bool((off <= tol).all()), float((off / tol).max())


def _call(api, c, **kw):
    return api.combine_norm(c["x"], c["o"], c["pos"], c["w"], post=c["post"], scale=c["scale"], pre=c["pre"], eps=c["eps"],
                            n_dtype=c["n_dtype"], **kw)


def _call_back(api, c, **kw):
    # (x stands for y)
    return api.combine_norm_backward(c["dy"], c["dn"], c["x"], c["o"], c["pos"], c["w"], post=c["post"], scale=c["scale"],
                                     pre=c["pre"], eps=c["eps"], **kw)


def _check(got, c):
    y, n = got
    want = _forward(c)
    if c["o"] is None:
        assert y is c["x"]
    else:
        assert y.dtype == c["x"].dtype
        _near_rows(y, *want[0])
    assert (n is None) == (c["pre"] is None)
    if n is not None:
        assert n.dtype == c["n_dtype"]
        _near_rows(n, *want[1])


def _check_back(got, c):
    want = _backward(c)
    got = dict(zip(("dx", "do", "dw", "dpost", "dscale", "dpre"), got))
    assert {n for n, t in got.items() if t is not None} == set(want)
    for n in want:
        (_near_rows if n in ("dx", "do") else _near)(got[n], *want[n])


SHAPES = [(1, 1, 8), (1, 2, 2048), (3, 8, 72), (67, 8, 264), (5, 3, 2056), (2, 6, 4104), (1, 8, 16384), (9, 4, 16384),
          (700, 2, 64), (400, 5, 520), (1031, 6, 1024), (160, 6, 4096), (330, 8, 8192), (320, 2, 12000)]


@pytest.mark.parametrize("T,k,H", SHAPES)
@pytest.mark.parametrize("types", [(F32, BF16, BF16), (F32, F32, F32), (BF16, BF16, F32), (BF16, F32, BF16)])
def test_matches_64_bits(cuda_lib, T, k, H, types):
    # (a norm behind one row takes its weight's effect away: that gradient is all rounding, and within its tolerance)
    c, st = _case(T, k, H, *types), cuda_lib.new_status()
    _check(_call(cuda_lib, c, status=st), c)
    c["do"] = None
    _check_back(_call_back(cuda_lib, c, status=st), c)
    assert int(st.item()) == 0


@pytest.mark.parametrize("T,k,H", [(3, 2, 136), (700, 8, 264)])
@pytest.mark.parametrize("kw", [
    dict(post=False), dict(scale=False), dict(pre=False), dict(post=False, scale=False, pre=False), dict(w=False),
    dict(pos=False), dict(pos=False, w=False, post=False), dict(rows=False), dict(post=False, scale=False),
])
def test_parts_left_out(cuda_lib, T, k, H, kw):
    if kw.get("w") is False and kw.get("pos") is False:
        k = 1  # (neither says how many rows a token has: one)
    c = _case(T, k, H, **kw)
    _check(_call(cuda_lib, c), c)
    _check_back(_call_back(cuda_lib, c), c)
    if c["pre"] is not None:  # y's own gradient missing
        c["dy"] = None
        _check_back(_call_back(cuda_lib, c), c)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("T,k,H", [(5, 2, 136), (700, 6, 264)])
def test_dropped_routes(cuda_lib, T, k, H, post):
    """Some routes have no row, some tokens none at all: they pass the stream
    on; the rows that nothing names stay as they were in do."""
    c = _case(T, k, H, drop=0.4, post=post)
    c["pos"][1] = -1
    c["pos"][-1] = -1
    c["o"][:] = torch.where(torch.isin(torch.arange(T * k, device=DEV), c["pos"]).unsqueeze(1), c["o"], float("nan"))
    got = _call(cuda_lib, c)
    c["o"] = torch.nan_to_num(c["o"], 0.0)
    _check(got, c)
    assert torch.equal(got[0][1], c["x"][1])
    do = torch.full_like(c["o"], -7.0)
    _check_back(_call_back(cuda_lib, c, do=do), c)


def test_rows_outside_count_as_dropped(cuda_lib):
    c = _case(40, 2, 72)
    bad = c["pos"].clone()
    bad[3, 0], bad[7, 1], bad[9, 0] = 80, -2, 2 ** 31 - 1
    c["pos"] = torch.where((bad < 0) | (bad >= 80), -1, bad)
    want = _call(cuda_lib, c)
    do = torch.full_like(c["o"], -7.0)
    back = _call_back(cuda_lib, c, do=do.clone())
    c["pos"] = bad
    for call, kw, ref in ((_call, {}, want), (_call_back, dict(do=do), back)):
        st = cuda_lib.new_status()
        got = call(cuda_lib, c, status=st, **kw)
        assert int(st.item()) == cuda_lib.MOE_DEV_BAD_ROUTE
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("T", [5, 700])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_with_its_token(cuda_lib, T, bad):
    c = _case(T, 3, 136)
    clean = _call(cuda_lib, c)
    back = _call_back(cuda_lib, c)
    c["o"][c["pos"][2, 1]] = bad
    c["x"][4] = bad
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[2] = keep[4] = False
    got = _call(cuda_lib, c)
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, clean))
    assert not bool(torch.isfinite(got[1][~keep]).any())
    got = _call_back(cuda_lib, c)
    rows = torch.ones(3 * T, dtype=torch.bool, device=DEV)
    rows[c["pos"][~keep].flatten().long()] = False
    assert torch.equal(got[0][keep], back[0][keep]) and torch.equal(got[1][rows], back[1][rows])
    assert torch.equal(got[2][keep], back[2][keep])


def test_no_tokens(cuda_lib):
    c = _case(0, 2, 72)
    y, n = _call(cuda_lib, c)
    assert y.shape == n.shape == (0, 72)
    dx, do, dw, *sums = _call_back(cuda_lib, c)
    assert dx.shape == do.shape == (0, 72) and dw.shape == (0, 2) and all(bool((s == 0).all()) for s in sums)


def test_no_rows_at_all(cuda_lib):
    """Every route dropped, an empty o: the stream passes on."""
    c = _case(6, 2, 72)
    c["o"], c["pos"] = c["o"][:0], torch.full_like(c["pos"], -1)
    y, n = _call(cuda_lib, c)
    assert torch.equal(y, c["x"]) and y is not c["x"]
    _check((y, n), c)
    _check_back(_call_back(cuda_lib, c), c)


def test_zero_rows_and_zero_streams(cuda_lib):
    c = _case(6, 2, 72)
    c["o"].zero_()
    c["x"][:3] = 0
    _check(_call(cuda_lib, c), c)
    _check_back(_call_back(cuda_lib, c), c)


@pytest.mark.parametrize("T,H", [(1, 2048), (67, 264), (3000, 520)])
def test_in_place_captured_and_on_another_stream(cuda_lib, T, H):
    c = _case(T, 4, H, x=BF16)
    first, back = _call(cuda_lib, c), _call_back(cuda_lib, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = _call(cuda_lib, c, stream=s) + _call_back(cuda_lib, c, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(other, first + back))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _call(cuda_lib, c) + _call_back(cuda_lib, c)
    keep = {n: t.clone() for n, t in c.items() if torch.is_tensor(t)}
    for n in ("x", "o", "w", "dy"):
        c[n].mul_(0.5)
    c["pos"].copy_(c["pos"].flip(0))
    g.replay()
    torch.cuda.synchronize()
    _check(out[:2], c)
    _check_back(out[2:], c)
    for n, t in keep.items():
        c[n].copy_(t)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, first + back))
    # in place: y into x, dx into dy
    x, dy = c["x"].clone(), c["dy"].clone()
    c2 = dict(c, x=x)
    y, n = _call(cuda_lib, c2, y=x)
    assert y is x and torch.equal(y, first[0]) and torch.equal(n, first[1])
    c2 = dict(c, dy=dy)
    got = _call_back(cuda_lib, c2, dx=dy)
    assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, back))


def test_two_streams_at_once(cuda_lib):
    cases = [_case(T, 3, 264, seed=T) for T in (1, 90, 2000)]
    want = [_call(cuda_lib, c) + _call_back(cuda_lib, c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [_call(cuda_lib, c, stream=s) + _call_back(cuda_lib, c, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("post", [True, False])
def test_gradients_against_differences(cuda_lib, post):
    """sum(y dy + n dn) moved along directions of every input: central
    differences of the formulas in 64 bits (step 2^-12: the third derivative's
    term is below 2^-18 of the magnitudes) against the kernel's gradients, each
    within the tolerances above."""
    c = _case(9, 3, 136, o=F32, n=F32, post=post)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    leaves = {n: c[n].double() for n in ("x", "o", "w", "post", "scale", "pre") if torch.is_tensor(c[n])}
    move = {n: torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64) * t.abs().mean() for n, t in leaves.items()}

    def loss(at):
        rows = at["o"][c["pos"].long()]
        z = (at["w"].unsqueeze(2) * rows).sum(1)
        b = z * _rms(z) * at["post"] if post else z
        y = at["x"] + at["scale"] * b
        return (y * c["dy"].double()).sum() + (y * _rms(y) * at["pre"] * c["dn"].double()).sum()

    back = dict(c, x=_call(cuda_lib, c)[0])  # y
    got = dict(zip(("x", "o", "w", "post", "scale", "pre"), _call_back(cuda_lib, back)))
    for n, v in move.items():
        t = 2.0 ** -12
        num = (loss({**leaves, n: leaves[n] + t * v}) - loss({**leaves, n: leaves[n] - t * v})) / (2 * t)
        m = (got[n].double() * v).abs().sum()
        assert abs(float(num - (got[n].double() * v).sum())) <= 2.0 ** -13 * float(m) + 2.0 ** -16, n


def test_offsets_past_32_bits(cuda_lib):
    """More than 2^31 elements in the rows."""
    R, H, T = 300_000, 8192, 500
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    c = _case(T, 2, H, o=BF16)
    o = torch.randn((R, H), generator=g, device=DEV, dtype=BF16)
    pos = (torch.randperm(T * 2, generator=g, device=DEV) + R - 2 * T).view(T, 2)
    small = dict(c, o=o[R - 2 * T:].clone(), pos=(pos - (R - 2 * T)).int())
    c.update(o=o, pos=pos.int())
    for a, b in zip(_call(cuda_lib, c), _call(cuda_lib, small)):
        assert torch.equal(a, b)
    got, want = _call_back(cuda_lib, c), _call_back(cuda_lib, small)
    assert torch.equal(got[1][R - 2 * T:], want[1])
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(got, want)) if i != 1)
    torch.cuda.empty_cache()


def test_the_most_tokens(cuda_lib):
    """2^22 tokens of one row, whose stream passes 2^31 elements."""
    T, H = cuda_lib.MAX_ROWS, 520
    x = torch.zeros((T, H), dtype=BF16, device=DEV)
    x[-3:] = 2.0
    pre = torch.full((H,), 1.5, device=DEV)
    _, n = cuda_lib.combine_norm(x, pre=pre)
    assert bool((n[-3:] == 1.5).all()) and bool((n[:-3] == 0).all())
    dx, _, _, _, _, dpre = cuda_lib.combine_norm_backward(None, n, x, pre=pre)
    # (2 / sqrt(4 + eps) rounds to 1 - 2^-23 or 1: three tokens of 1.5 each)
    assert bool(((dpre - 4.5).abs() <= 4.5 * 2.0 ** -20).all()) and bool((dx[:-3] == 0).all())
    torch.cuda.empty_cache()
