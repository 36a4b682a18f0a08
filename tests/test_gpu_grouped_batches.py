"""The grouped products on batches of more tokens than the router's kernels
take (MAX_B): the offsets then come from a grouping made with torch."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _group(ids, E):
    """-> (offsets, route_idx) as group_by_expert returns them, for any number of tokens."""
    e = ids.flatten().long()
    offsets = torch.cat([e.new_zeros(1), torch.bincount(e, minlength=E).cumsum(0)]).int()
    return offsets, e.argsort(stable=True).int()


@pytest.mark.parametrize("B,k,E", [(1, 1, 1), (64, 4, 40), (1024, 8, 256)])
def test_the_grouping_is_group_by_expert_s(cuda_lib, B, k, E):
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    ids = torch.rand((B, E), generator=g, device=DEV).topk(k, dim=1).indices.int()
    want = cuda_lib.group_by_expert(ids, E)
    for a, b in zip(_group(ids, E), want):
        assert torch.equal(a, b)


def test_a_batch_of_more_tokens_than_the_router_takes(cuda_lib):
    B, k, E, N, K = 3000, 2, 10, 136, 264
    assert B > cuda_lib.MAX_B
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    ids = torch.rand((B, E), generator=g, device=DEV).topk(k, dim=1).indices.int()
    with pytest.raises(cuda_lib.MoeError):
        cuda_lib.group_by_expert(ids, E)
    x = torch.randn((B, K), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((E, N, K), generator=g, device=DEV).to(torch.bfloat16)
    offsets, route_idx = _group(ids, E)
    route_idx = route_idx.long()
    xs = x[route_idx // k]
    y = cuda_lib.grouped_gemm(xs, w, offsets)
    we = w[ids.flatten()[route_idx].long()].double()
    ref = torch.einsum("rk,rnk->rn", xs.double(), we)
    mag = torch.einsum("rk,rnk->rn", xs.double().abs(), we.abs())
    assert bool(((y.double() - ref).abs() <= (K + 1) * 2.0 ** -23 * mag).all())
