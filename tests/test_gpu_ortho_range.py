"""What orthogonalisation (moe_orthogonalize) loses where that would show
most."""
import math

import pytest
import torch

import test_gpu_ortho as ortho

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("N,K", [(16384, 16256), (16384, 16258), (16383, 16257), (16383, 16259)])
@pytest.mark.parametrize("v", [0.7, 1.45, 1.1, 0.9])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_norm_of_many_equal_values(cuda_lib, N, K, v, dtype):
    """X = G / |G|_F alone: 1 / sqrt(N K) in bf16, whatever the value.  The
    sizes put it 2.3e-5 above or 3.8e-5 below the middle of two bf16 values, so
    that a norm which a long sum of squares left off by more shows up in every
    value of the result.  Allowed is 2^-17 = 7.6e-6: 2^-19 of the norm and
    half of fp16's smallest step, 2^-25, in what 22 bits leave of 2^-6."""
    g = torch.full((N, K), v, device=DEV).to(dtype)
    want = 1.0 / math.sqrt(N * K)
    got = cuda_lib.orthogonalize(g, steps=1, coeffs=(1.0, 0.0, 0.0), eps=0.0)
    lo, hi = (torch.tensor(want * (1 + s * 2.0 ** -17), dtype=torch.float64).to(BF16) for s in (-1, 1))
    assert bool(lo == hi)
    assert bool((got == lo.to(DEV)).all()), (float(got[0, 0]), float(lo))
    del g, got
    torch.cuda.empty_cache()
