"""A routing whose balance bias changes between calls, against the float64 form."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


def test_the_bias_changes(dev):
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(1)
    M, E, k = 40, 64, 6
    kw = dict(score="sigmoid", n_groups=8, topk_groups=3, group_top=2)
    lg = torch.randn(M, E, generator=g)
    d = lg.to(dev)
    b = [torch.randn(E, generator=g) * 0.5 for _ in range(4)]
    r = moe.Routing(bias=b[0].to(dev), **kw)

    def same(bias):
        ids, _ = moe.moe_route_grouped(d, k, r)
        assert torch.equal(ids.cpu(), ref.route(lg, k, bias=bias, **kw)[0])

    same(b[0])
    r.bias.copy_(b[1])        # in place
    same(b[1])
    r.bias = b[2].to(dev)     # another tensor
    same(b[2])
    r.bias.data = b[3].to(dev)  # the same tensor, another storage
    same(b[3])
    r.bias = None
    same(None)


def test_the_bias_changes_under_a_graph(dev):
    """A captured call keeps the tensor it was captured with: in place changes
    reach its replays, another tensor only later calls."""
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(2)
    M, E, k = 17, 32, 4
    lg = torch.randn(M, E, generator=g)
    d = lg.to(dev)
    b = [torch.randn(E, generator=g) * 0.5 for _ in range(3)]
    first = b[0].to(dev)
    r = moe.Routing("sigmoid", first)
    ids = torch.empty(M, k, dtype=torch.int32, device=dev)
    w = torch.empty(M, k, device=dev)
    moe.moe_route_grouped(d, k, r, topk_ids=ids, topk_weights=w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_route_grouped(d, k, r, topk_ids=ids, topk_weights=w)
    want = [ref.route(lg, k, score="sigmoid", bias=t)[0] for t in b]
    r.bias = b[1].to(dev)
    for t, rid in ((b[0], want[0]), (b[2], want[2]), (b[0], want[0])):
        first.copy_(t)
        ids.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu(), rid)
        eager, _ = moe.moe_route_grouped(d, k, r)
        assert torch.equal(eager.cpu(), want[1])
