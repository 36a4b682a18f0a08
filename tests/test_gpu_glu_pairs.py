"""The gated unit and its gradient where their tiles are those of CTA pairs (from
256 rows a segment on average, 512 to fp32, 144 for the gradient), and one row
to either side of where the pairs begin.
Tolerances as in test_gpu_glu.py."""
import pytest
import torch

import test_gpu_glu as glu

pytestmark = pytest.mark.gpu

# ragged ends and empty segments, widths that end inside a tile, a contraction of several accumulators
SHAPES = [([1500, 0, 700], 392, 1000), ([513, 600, 1201], 72, 264), ([1100, 1], 264, 4104), ([511], 136, 200), ([512], 136, 200),
          ([143], 136, 200), ([144], 136, 200), ([255], 136, 200), ([256], 136, 200), ([200, 400, 0, 470], 392, 1000)]


@pytest.mark.parametrize("act", glu.ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,I,H", SHAPES)
def test_matches_64_bit_loops(cuda_lib, counts, I, H, dtype, act):
    c, st = glu._case(counts, I, H), cuda_lib.new_status()
    got = cuda_lib.grouped_glu(c["x"], c["w"], c["off"], act=act, keep=True, out_dtype=dtype, status=st)
    glu._check_forward(got, c, act)
    glu._check_backward(cuda_lib.grouped_glu_backward(c["dy"], c["down"], c["gu"], c["off"], act=act, status=st), c, act)
    assert int(st.item()) == 0
