"""A training step of one pre-norm MoE layer as a user writes it with the
library's operators: norm, routing, the experts' block, the join with the next
norm, every gradient, and the experts' update orthogonalised.

Against autograd through the same formulas in 64 bits, on the routing that the
library chose.  Each of the values that pass from one operator to the next in
bf16 (the normed input, h, the rows o, do, dgu) is off by half a step, 2^-8 of
it at most and independently of the others; a gradient sums hundreds of them,
so that its 2-norm is off by at most 2^-8 for each of the five."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,H,I,E,k,act", [(96, 256, 128, 12, 3, "silu"), (515, 264, 72, 8, 2, "gelu"), (700, 128, 520, 5, 4, "silu")])
def test_a_training_step(cuda_lib, T, H, I, E, k, act):
    api = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, router = r(T, H), (r(E, H) * H ** -0.5).bfloat16()
    gate_up, down = (r(E, 2 * I, H) * H ** -0.5).bfloat16(), (r(E, H, I) * I ** -0.5).bfloat16()
    pre, post, scale, nxt = 1 + 0.1 * r(H), 1 + 0.1 * r(H), 0.5 + 0.1 * r(H), 1 + 0.1 * r(H)
    dy, dn = r(T, H) * 0.1, (r(T, H) * 0.1).bfloat16()

    # forward
    _, n = api.combine_norm(x, pre=pre)
    ids, w, _ = api.route(n, router, k)
    off, ridx, _, _ = api.group_by_expert(ids, E)
    pos = torch.empty_like(ridx)
    pos[ridx.long()] = torch.arange(T * k, dtype=torch.int32, device=DEV)
    pos = pos.view(T, k)
    xs = n[ridx.long() // k]
    h, gu = api.grouped_glu(xs, gate_up, off, act=act, keep=True)
    o = api.grouped_gemm(h, down, off, out_dtype=torch.bfloat16)
    y, n2 = api.combine_norm(x, o, pos, w, post=post, scale=scale, pre=nxt)
    # backward
    dx, do, dw, dpost, dscale, dnxt = api.combine_norm_backward(dy, dn, y, o, pos, w, post=post, scale=scale, pre=nxt)
    dgu, h2 = api.grouped_glu_backward(do, down, gu, off, act=act)
    ddown = api.grouped_gemm_dw(do, h2, off)
    dgate_up = api.grouped_gemm_dw(dgu, xs, off)
    dxs = api.grouped_gemm_dx(dgu, gate_up, off)
    dnorm = torch.zeros((T, H), device=DEV).index_add_(0, ridx.long() // k, dxs)
    dx0, _, _, _, _, dpre = api.combine_norm_backward(dx, dnorm, x, pre=pre)
    update = api.orthogonalize(dgate_up)

    # the same in 64 bits
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    X, G, D, W, P, Q, S, N2 = (leaf(t) for t in (x, gate_up, down, w, pre, post, scale, nxt))
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    n64 = rms(X) * P
    z = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        a = n64[t] @ G[e].T
        gate = a[:, :I]
        unit = torch.nn.functional.silu(gate) if act == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
        z = z.index_add(0, t, W[t, j].unsqueeze(1) * ((unit * a[:, I:]) @ D[e].T))
    y64 = X + S * (rms(z) * Q)
    out64 = rms(y64) * N2
    ((y64 * dy.double()).sum() + (out64 * dn.double()).sum()).backward()

    def near(got, want, steps):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= steps * 2.0 ** -8, rel

    near(y, y64.detach(), 3)
    near(n2, out64.detach(), 4)
    near(dx0, X.grad, 5)
    for got, want in ((dgate_up, G), (ddown, D), (dw, W), (dpre, P), (dpost, Q), (dscale, S), (dnxt, N2)):
        near(got, want.grad, 5)
    # the update: the recurrence in 64 bits on the same gradient (its roundings: test_gpu_ortho.py)
    u = dgate_up.double()
    u = u.mT if 2 * I > H else u
    u = u / (u.flatten(1).norm(dim=1).view(-1, 1, 1) + 1e-7)
    for _ in range(5):
        m = u @ u.mT
        u = 3.4445 * u + (-4.7750 * m + 2.0315 * m @ m) @ u
    near(update, u.mT if 2 * I > H else u, 2)
