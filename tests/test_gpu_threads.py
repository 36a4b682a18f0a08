"""Host threads that call the library at the same time, each on a stream of its
own: ctypes releases the interpreter's lock during a call, so that their calls
interleave inside the library."""
import threading

import pytest
import torch

import test_gpu_join as join

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _together(calls, times):
    """Every call `times` times in a thread of its own, all at once -> the last results, the errors."""
    streams = [torch.cuda.Stream() for _ in calls]
    results, errors, ready = [None] * len(calls), [], threading.Barrier(len(calls))
    torch.cuda.synchronize()

    def work(i):
        ready.wait()
        try:
            for _ in range(times):
                results[i] = calls[i](streams[i])
        except Exception as e:  # noqa: BLE001
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return results, errors


def _calls_of(api, monkeypatch, name, run):
    """What the binding passes to the C entry `name` in each call that run() makes."""
    calls, lib = [], api._lib

    class Keep:
        def __getattr__(self, n):
            f = getattr(lib, n)
            return (lambda *args: calls.append(args) or f(*args)) if n == name else f

    with monkeypatch.context() as m:
        m.setattr(api, "_lib", Keep())
        kept = run()
    return calls, kept


def _again(api, name, calls, times):
    """Each of the C calls `times` times in a thread of its own, so that they meet inside the entry -> their codes."""
    f, codes = getattr(api._lib, name), [set() for _ in calls]

    def work(i):
        for _ in range(times):
            codes[i].add(f(*calls[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return codes


@pytest.mark.parametrize("widths", [(8200, 16384), (12000, 16384), (3000, 4096)])
def test_gradients_of_the_join_of_different_widths(cuda_lib, monkeypatch, widths):
    """One kernel whose shared memory depends on the width and on how many
    vectors have a gradient."""
    cases = [join._case(2, 2, H, F32, BF16, BF16, scale=s, seed=H) for H in widths for s in (True, False)]
    streams, spaces = [torch.cuda.Stream() for _ in cases], [torch.empty(1 << 20, dtype=torch.uint8, device=DEV) for _ in cases]
    calls, got = _calls_of(cuda_lib, monkeypatch, "moe_combine_norm_backward",
                           lambda: [join._call_back(cuda_lib, c, stream=s, workspace=w)
                                    for c, s, w in zip(cases, streams, spaces)])
    torch.cuda.synchronize()
    want = [[None if t is None else t.clone() for t in ts] for ts in got]
    for ts in got:
        for t in ts:
            if t is not None:
                t.zero_()
    codes = _again(cuda_lib, "moe_combine_norm_backward", calls, 4000)
    assert codes == [{cuda_lib.MOE_OK}] * len(calls), codes
    for a, b in zip(got, want):
        assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


def test_experts_of_different_widths(cuda_lib, monkeypatch):
    """The same of the experts' kernels (on one stream)."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    B, I, E, k = 4, 64, 4, 2
    ids = torch.tensor([[0, 1], [1, 2], [3, 0], [2, 3]], dtype=torch.int32, device=DEV)
    w = torch.full((B, k), 0.5, device=DEV)
    group = cuda_lib.group_by_expert(ids, E)
    cases = [(r(B, H), r(E, 2 * I, H).to(BF16), r(E, H, I).to(BF16), cuda_lib.new_workspace(B, H, I, E, k, DEV))
             for H in (4096, 6400)]
    calls, got = _calls_of(cuda_lib, monkeypatch, "moe_expert_forward",
                           lambda: [cuda_lib.expert_forward(x, g, d, ids, w, group, flags=cuda_lib.MOE_F_NO_TC, workspace=ws)
                                    for x, g, d, ws in cases])
    want = [t.clone() for t in got]
    codes = _again(cuda_lib, "moe_expert_forward", calls, 3000)
    assert codes == [{cuda_lib.MOE_OK}] * len(calls), codes
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_wide_and_narrow_gradients_in_one_capture(cuda_lib):
    cases = [join._case(2, 2, H, F32, BF16, BF16, scale=s, seed=H) for H, s in ((16384, True), (8200, False), (12000, True))]
    want = [join._call_back(cuda_lib, c) for c in cases]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [join._call_back(cuda_lib, c) for c in cases]
    join._call_back(cuda_lib, cases[1])
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all((p is None and q is None) or torch.equal(p, q) for p, q in zip(a, b))


def test_all_operators_at_once(cuda_lib):
    """Both tile widths of the products, and the other operators, each in its own thread."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV, dtype=BF16)  # noqa: E731
    off = torch.tensor([0, 40, 40, 300], dtype=torch.int32, device=DEV)
    x, w, down, gu = r(300, 136), r(3, 528, 136), r(3, 136, 264), r(300, 528)
    g, big = r(3, 72, 200), r(40, 260, 300)
    c = join._case(70, 2, 520)
    calls = [lambda s: cuda_lib.grouped_glu(x, w, off, keep=True, stream=s),
             lambda s: cuda_lib.grouped_glu_backward(x, down, gu, off, stream=s),
             lambda s: join._call(cuda_lib, c, stream=s),
             lambda s: join._call_back(cuda_lib, c, stream=s),
             lambda s: (cuda_lib.orthogonalize(g, stream=s),),
             lambda s: (cuda_lib.orthogonalize(big, stream=s),)]
    want = [f(None) for f in calls]
    got, errors = _together(calls, 100)
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
