"""Routing weights from scores that float32 cannot hold, against the float64 form.

A score below float32's normals is not a weight of 0: a factor, or the sum it is
divided by, brings it back.  Weights are within (32 + span) half-steps of 2^-24 as
in the other router tests (a float32 sum may be left in the denominator), and half
the smallest subnormal step, 2^-150."""
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


def rows():
    """[n, 32] logits: chosen scores from 1e-27 down to below 2^-149, alone, together
    and beside larger ones; masked experts and whole masked rows among them."""
    inf = float("inf")
    g = torch.Generator().manual_seed(3)
    lg = torch.full((12, 32), -400.0) - torch.rand(12, 32, generator=g) * 50
    lg[0, :8] = torch.linspace(-60, -88, 8)      # float32 holds each, some in subnormals
    lg[1, :8] = torch.linspace(-86, -103, 8)     # subnormal
    lg[2, :8] = torch.linspace(-104, -160, 8)    # nothing that float32 holds
    lg[3, :8] = torch.linspace(3, -200, 8)
    lg[4, :4] = torch.tensor([-68.0, -89.0, -95.0, -150.0])
    lg[5, 2:] = -inf                             # two experts left, both far below
    lg[5, :2] = torch.tensor([-90.0, -91.0])
    lg[6] = -inf
    lg[7, 5] = inf
    lg[8] = -89.5
    lg[9, ::2] = torch.linspace(-80, -120, 16)
    lg[10, :8] = torch.linspace(40, -89, 8)
    lg[11, :8] = torch.linspace(-88.6, -88.8, 8)
    return lg


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scale", [1.0, 1e30, -2.5e37])
@pytest.mark.parametrize("groups", [dict(), dict(n_groups=4, topk_groups=2, group_top=2)])
def test_small_weights(dev, score, renormalize, scale, groups):
    import moe_layer_topk_amd as moe
    lg = rows()
    kw = dict(score=score, renormalize=renormalize, scale=scale, **groups)
    ids, w = moe.moe_route_grouped(lg.to(dev), 8, moe.Routing(**kw))
    rid, rw = ref.route(lg, 8, **kw)
    assert torch.equal(ids.cpu(), rid)
    fin = torch.where(torch.isfinite(lg), lg, torch.zeros_like(lg)).double()
    span = (fin.amax(1, keepdim=True) - fin.amin(1, keepdim=True)).clamp_max(104.0)
    assert bool(torch.isfinite(w).all())
    err = (w.cpu().double() - rw).abs()
    tol = (32 + span) * 2.0 ** -24 * rw.abs() + 2.0 ** -150
    assert bool((err <= tol).all()), (err / tol).amax(1)


@pytest.mark.parametrize("M", [1, 12])
def test_small_weights_of_a_layer(dev, M):
    """The same weights from the router inside a layer's launches."""
    import moe_layer_topk_amd as moe
    from test_gpu_block_fp8 import weights
    E, k, H, I = 32, 8, 128, 128
    w1, s1 = (t.to(dev) for t in weights(E, 2 * I, H, 1))
    w2, s2 = (t.to(dev) for t in weights(E, H, I, 2))
    x = torch.randn(M, H, generator=torch.Generator().manual_seed(1)).bfloat16().to(dev)
    for lg in ([rows()] if M > 1 else rows().split(1)):
        r = moe.Routing("sigmoid", renormalize=False, scale=1e30)
        ids = torch.empty(M, k, dtype=torch.int32, device=dev)
        w = torch.empty(M, k, device=dev)
        moe.fused_moe_grouped(x, lg.contiguous().to(dev), w1, w2, k, r, w1_scale=s1, w2_scale=s2, topk_ids=ids, topk_weights=w)
        rid, rw = ref.route(lg, k, score="sigmoid", renormalize=False, scale=1e30)
        assert torch.equal(ids.cpu(), rid)
        assert bool(((w.cpu().double() - rw).abs() <= 136 * 2.0 ** -24 * rw + 2.0 ** -150).all())
