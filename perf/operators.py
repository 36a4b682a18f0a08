"""The grouped-product operators, case by case: inputs, the plain form of each
operator in elementary torch operations, the library's calls, and the same
results in 64 bits.

Operators (rows r of x grouped by expert: segment e is rows
offsets[e] .. offsets[e+1]-1):

  gemm    y[r, :] = w[e] x[r, :]             x [R, K], w [E, N, K] bf16
  dx      dx[r, :] = w[e]^T dy[r, :]         dy [R, N]
  dw      dw[e] = sum_r dy[r, :] x[r, :]^T   [E, N, K]
  quant   x -> NVFP4 codes, block scales and scale, and back to values
  gemm4   y[r, :] = w[e] x[r, :] with both operands in NVFP4

``own`` selects the library's kernels (True) or the plain form (False).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token, top-2 of 128 experts: the call's latency
        dict(name="gemm one token", op="gemm", R=2, N=1536, K=2048, E=128, k=2, skew=False, out="f32"),
        # a decode batch of 64 tokens, top-8 of 256: every expert's weights stream once
        dict(name="gemm decode batch", op="gemm", R=512, N=1536, K=2048, E=256, k=8, skew=False, out="bf16"),
        # the down projection of 128 tokens with a few popular experts
        dict(name="gemm skewed down", op="gemm", R=768, N=2048, K=768, E=256, k=6, skew=True, out="f32"),
        # a training batch's gate/up projection: about a thousand rows an expert
        dict(name="gemm training", op="gemm", R=65536, N=1536, K=2048, E=64, k=8, skew=False, out="bf16"),
        # the input gradient of a small fine-tuning batch, about 16 rows an expert
        dict(name="dx small batch", op="dx", R=4096, N=4096, K=1536, E=256, k=8, skew=False, out="bf16"),
        # the input gradient of the training batch
        dict(name="dx training", op="dx", R=65536, N=1536, K=2048, E=64, k=8, skew=False, out="bf16"),
        # the weight gradient of a few hundred rows, kept in 32 bits for accumulation
        dict(name="dw few rows", op="dw", R=515, N=2048, K=768, E=128, k=2, skew=True, out="f32"),
        # the weight gradient of the training batch
        dict(name="dw training", op="dw", R=65536, N=1536, K=2048, E=64, k=8, skew=False, out="bf16"),
        # a layer's down weights into NVFP4, and back (what a model with such weights computes with)
        dict(name="quant weights", op="quant", G=256, rows=2048, cols=768, type="bf16", out="bf16"),
        # the activations of a prompt into NVFP4, one scale a token
        dict(name="quant tokens", op="quant", G=4099, rows=1, cols=2048, type="f32", out="f32"),
        # a decode batch of 4 tokens on NVFP4 experts
        dict(name="gemm4 decode", op="gemm4", R=32, N=1536, K=2048, E=256, k=8, skew=False, out="f32"),
        # a large prompt batch on NVFP4 experts
        dict(name="gemm4 prefill", op="gemm4", R=65536, N=1536, K=2048, E=64, k=8, skew=False, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "dx", "dw", "quant", "gemm4"])
    if op == "quant":
        cols = 32 * _log(rng, 2, 256)
        if rng.random() < 0.5:
            G, rows = _log(rng, 1, 65536), 1
        else:
            G, rows = _log(rng, 1, 256), _log(rng, 16, 4096)
        while G * rows * cols > 256 * 2048 * 768:
            G = max(1, G // 2)
            cols = max(64, cols // 64 * 32)
        return dict(op=op, G=G, rows=rows, cols=cols, type=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    step = 32 if op == "gemm4" else 8
    N, K = (step * _log(rng, 64 // step, 4096 // step) for _ in range(2))
    E, R = _log(rng, 1, 256), _log(rng, 1, 65536)
    while E * N * K > 256 * 1536 * 2048:
        E = max(1, E // 2)
    while R * N * K > 65536 * 1536 * 2048:
        R = max(1, R // 2)
    return dict(op=op, R=R, N=N, K=K, E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])), skew=rng.random() < 0.3,
                out=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs
def _routes(case, g):
    """Rows a segment of a step with k experts a token: the k largest of random logits (with a Zipf-like bias where skewed)."""
    R, E, k = case["R"], case["E"], case["k"]
    logits = torch.randn((-(-R // k), E), generator=g, device="cuda")
    if case["skew"]:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
        logits += 2.0 * torch.log(rank ** -1.1)
    ids = logits.topk(k, dim=1).indices.flatten()[:R]
    return torch.bincount(ids, minlength=E)


def _normal(shape, sigma, g, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _plan(counts):
    """The segments as a padded batch: which rows of x (R: a row of zeros) fill [active experts, longest], and where each row went."""
    counts = counts.tolist()
    R, off = sum(counts), np.concatenate([[0], np.cumsum(counts)])
    active = [e for e, c in enumerate(counts) if c]
    cap = max(counts)
    at = np.full((len(active), cap), R, np.int64)
    back = np.empty(R, np.int64)
    for u, e in enumerate(active):
        at[u, :counts[e]] = np.arange(off[e], off[e + 1])
        back[off[e]:off[e + 1]] = u * cap + np.arange(counts[e])
    t = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    return dict(offsets=t(off.astype(np.int32)), at=t(at), back=t(back), active=t(np.array(active, np.int64)),
                counts=counts)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], dict(case=case)
    if op == "quant":
        # weights ~ N(0, 0.02) a matrix; tokens of differing magnitude, as after a few layers
        rows, per_row = case["rows"], case["rows"] == 1
        shape = (case["G"], case["cols"]) if per_row else (case["G"], rows, case["cols"])
        x = torch.randn(shape, generator=g, device="cuda")
        x = x * torch.exp(torch.randn((case["G"], 1), generator=g, device="cuda")) if per_row else x * 0.02
        s["x"] = x.to(TYPES[case["type"]])
        return s
    R, N, K, E = (case[n] for n in ("R", "N", "K", "E"))
    s.update(_plan(_routes(case, g)))
    if op in ("gemm", "dw", "gemm4"):
        s["x"] = _normal((R, K), 1.0, g)
    if op in ("dx", "dw"):
        s["dy"] = _normal((R, N), 0.01, g)
    if op in ("gemm", "dx", "gemm4"):
        s["w"] = _normal((E, N, K), 0.02, g)
    if op == "gemm4":
        s["xq"], s["wq"] = _quantize(s.pop("x")), _quantize(s.pop("w"))
    return s


# -------------------------------------------------------------- plain forms
def _padded(t, s):
    t = t.float()
    return torch.cat([t, t.new_zeros(1, t.shape[1])])[s["at"]]


def _back(p, s):
    return p.flatten(0, 1)[s["back"]]


def _quantize(x):
    """NVFP4 of x: one scale gs a matrix of x [G, rows, cols], or a row of x [G, cols]; one E4M3 scale per 16 elements; E2M1 codes.

    gs = amax / (448 * 6), rounded up to 8 significant bits (2^-100 at least); block scale = E4M3 nearest to block amax / (6 gs);
    code = E2M1 nearest to x / (block scale * gs), both ties to even.  Products of the scales are exact in 32 bits."""
    f = x.float()
    amax = f.abs().amax(dim=tuple(range(1, f.dim())))
    m, e = torch.frexp(amax.double() / 2688.0)
    gs = torch.ldexp(torch.ceil(m * 256.0) / 256.0, e).clamp(min=2.0 ** -100).float()
    b = f.unflatten(-1, (-1, 16))
    g = gs.view(-1, *[1] * (f.dim() - 1))
    bs = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    scale = (bs.float() * g).unsqueeze(-1)
    a = torch.where(scale > 0, b / scale, 0.0)
    neg, a = a < 0, a.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += (neg & (code > 0)).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), bs.view(torch.uint8), gs


def _values(q, bs):
    """E2M1 codes times their E4M3 block scales, in 32 bits (exact)."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    e, f = ((code & 7) >> 1).float(), (code & 1).float()
    v = torch.where(e > 0, (1.0 + 0.5 * f) * torch.exp2(e - 1.0), 0.5 * f)
    v = torch.where(code > 7, -v, v)
    return (v.unflatten(-1, (-1, 16)) * bs.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _plain(s):
    case = s["case"]
    op, out = case["op"], TYPES[case["out"]]
    if op == "quant":
        q, bs, gs = _quantize(s["x"])
        v = _values(q, bs) * gs.view(-1, *[1] * (s["x"].dim() - 1))
        return v.to(out), bs.view(torch.float8_e4m3fn), gs
    if op == "gemm":
        return _back(torch.bmm(_padded(s["x"], s), s["w"][s["active"]].float().mT), s).to(out)
    if op == "dx":
        return _back(torch.bmm(_padded(s["dy"], s), s["w"][s["active"]].float()), s).to(out)
    if op == "dw":
        dw = torch.zeros((case["E"], case["N"], case["K"]), dtype=out, device="cuda")
        dw[s["active"]] = torch.bmm(_padded(s["dy"], s).mT, _padded(s["x"], s)).to(out)
        return dw
    (xq, xbs, xgs), (wq, wbs, wgs) = s["xq"], s["wq"]
    a = s["active"]
    y = torch.bmm(_padded(_values(xq, xbs), s), _values(wq[a], wbs[a]).mT) * wgs[a].view(-1, 1, 1)
    return (_back(y, s) * xgs.unsqueeze(1)).to(out)


# --------------------------------------------------------- the library's own
def _library(s):
    from moe_decode_layer_gemv_gb300 import api
    case = s["case"]
    op, out = case["op"], TYPES[case["out"]]
    if op == "quant":
        q, bs, gs = api.quantize_nvfp4(s["x"])
        return api.dequantize_nvfp4(q, bs, gs, out_dtype=out), bs.view(torch.float8_e4m3fn), gs
    if op == "gemm":
        return api.grouped_gemm(s["x"], s["w"], s["offsets"], out_dtype=out)
    if op == "dx":
        return api.grouped_gemm_dx(s["dy"], s["w"], s["offsets"], out_dtype=out)
    if op == "dw":
        return api.grouped_gemm_dw(s["dy"], s["x"], s["offsets"], out_dtype=out)
    return api.grouped_gemm_nvfp4(*s["xq"], *s["wq"], s["offsets"], out_dtype=out)


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------- floors
def work(case):
    size = {"bf16": 2, "f32": 4}
    out = size[case["out"]]
    if case["op"] == "quant":
        n, cols = case["G"] * case["rows"] * case["cols"], case["cols"]
        coded = n / 2 + n / 16 + 4 * case["G"]
        # read x, write the codes; read them again, write the values
        return {"bytes": n * (size[case["type"]] + out) + 2 * coded, "flops": 4.0 * n}
    R, N, K, E = (case[n] for n in ("R", "N", "K", "E"))
    # experts with a row, as uniform routing has them; under skewed routing the popular ones alone
    tokens = -(-R // case["k"])
    if case["skew"]:
        p = np.arange(1, E + 1) ** -2.2
        active = float(np.sum(1.0 - (1.0 - np.minimum(1.0, case["k"] * p / p.sum())) ** tokens))
    else:
        active = E * (1.0 - (1.0 - case["k"] / E) ** tokens)
    active = max(1.0, min(active, R, E))
    flops = 2.0 * R * N * K
    if case["op"] == "gemm4":
        return {"bytes": (R * K + active * N * K) * 0.5625 + 4 * (R + active) + out * R * N, "flops": flops}
    if case["op"] == "dw":
        return {"bytes": 2 * R * (N + K) + out * E * N * K, "flops": flops}
    i, o = (K, N) if case["op"] == "gemm" else (N, K)
    return {"bytes": 2 * R * i + 2 * active * N * K + out * R * o, "flops": flops}


# ------------------------------------------------------------------ 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3():
    """The finite magnitudes of E4M3 (bias 7, three mantissa bits, largest 448), ascending by code."""
    return [(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127]


def _nearest(a, table):
    """The index of the table's value nearest to a, ties to the even index."""
    t = torch.tensor(table, dtype=torch.float64, device=a.device)
    mid = (t[1:] + t[:-1]) / 2
    lo = torch.bucketize(a, mid)              # midpoints below a
    hi = torch.bucketize(a, mid, right=True)  # ... and those equal to it
    return torch.where(lo % 2 == 0, lo, hi)


def _exact_quant(x):
    """One matrix or row group [rows, cols] -> (values, block scales, scale)."""
    a = x.double()
    top = float(a.abs().max())
    gs = 0.0
    if top > 0:
        m, e = math.frexp(top / 2688.0)
        gs = math.ldexp(math.ceil(m * 256), e - 8)
    gs = max(gs, 2.0 ** -100)
    b = a.reshape(a.shape[0], -1, 16)
    bs = torch.tensor(_e4m3(), dtype=torch.float64, device=a.device)[_nearest(b.abs().amax(-1) / (6 * gs), _e4m3())]
    s = bs.unsqueeze(-1) * gs
    q = torch.where(s > 0, b.abs() / torch.where(s > 0, s, 1.0), 0.0)
    v = torch.tensor(_E2M1, dtype=torch.float64, device=a.device)[_nearest(q, _E2M1)] * s
    return torch.where(b < 0, -v, v).reshape(a.shape), bs, gs


def _exact_values(q, bs, gs):
    lut = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=q.device)
    v = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.float64, device=q.device)
    v[..., 0::2] = lut[(q % 16).long()]
    v[..., 1::2] = lut[(q // 16).long()]
    s = torch.tensor(_e4m3(), dtype=torch.float64, device=q.device)[bs.long()]
    return v * s.repeat_interleave(16, dim=-1) * gs.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"]
        if x.dim() == 2:
            if x.shape[0] > 8192:
                return None
        v = torch.empty(x.shape, dtype=torch.float64 if x.numel() < 1 << 28 else torch.float32, device=x.device)
        bs = torch.empty((*x.shape[:-1], x.shape[-1] // 16), dtype=torch.float32, device=x.device)
        gs = torch.empty(x.shape[0], dtype=torch.float64, device=x.device)
        for i in range(x.shape[0]):
            vi, bi, gs[i] = _exact_quant(x[i].reshape(-1, x.shape[-1]))
            v[i], bs[i] = vi.reshape(x[i].shape), bi.reshape(bs[i].shape)
        return v, bs, gs
    R, N, K, E = (case[n] for n in ("R", "N", "K", "E"))
    if case["op"] == "dw":
        out = torch.zeros((E, N, K), dtype=torch.float32 if E * N * K > 1 << 28 else torch.float64, device="cuda")
    else:
        out = torch.zeros((R, K if case["op"] == "dx" else N), dtype=torch.float64, device="cuda")
    r = 0
    for e, n in enumerate(s["counts"]):
        if n == 0:
            continue
        seg = slice(r, r + n)
        if case["op"] == "gemm":
            out[seg] = s["x"][seg].double() @ s["w"][e].double().T
        elif case["op"] == "dx":
            out[seg] = s["dy"][seg].double() @ s["w"][e].double()
        elif case["op"] == "dw":
            out[e] = s["dy"][seg].double().T @ s["x"][seg].double()
        else:
            (xq, xbs, xgs), (wq, wbs, wgs) = s["xq"], s["wq"]
            out[seg] = _exact_values(xq[seg], xbs[seg], xgs[seg].unsqueeze(1)) @ _exact_values(wq[e], wbs[e], wgs[e]).T
        r += n
    return out
