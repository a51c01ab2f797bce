"""Per-expert scales of e4m3 weights in the shapes that a reduction over an
expert's matrix leaves: [E] and [E, 1, 1] are the same layer, bit for bit."""
from dataclasses import replace

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


@pytest.mark.parametrize("M", [1, 5, 70])
def test_scales_that_kept_their_dimensions(dev, M):
    import moe_layer_topk_amd as moe
    from workloads import CONFIGS, layer_batch, layer_weights
    E, k, H, I = 4, 2, 512, 256
    cfg = replace(CONFIGS["fp8_e4m3"], E=E, topk=k, H=H, I=I, router="normal")
    w = layer_weights(cfg, dev)
    b = layer_batch(cfg, M, dev)
    flat = dict(x_scale=b["x_scale"], w1_scale=w["w1_scale"].view(E), w2_scale=w["w2_scale"].view(E))
    kept = dict(x_scale=b["x_scale"], w1_scale=w["w1_scale"].view(E, 1, 1), w2_scale=w["w2_scale"].view(E, 1, 1))
    args = (b["x"], b["logits"], w["w1"], w["w2"], k)
    for f in (moe.fused_moe, moe.fused_moe_noalloc, lambda *a, **kw: moe.fused_moe_grouped(*a, moe.Routing(), **kw)):
        assert torch.equal(f(*args, **kept), f(*args, **flat))
    rw = torch.randn(E, H, generator=torch.Generator().manual_seed(1)).to(dev) * 0.1
    out, lg = moe.fused_moe_router(b["x"], rw, w["w1"], w["w2"], k, **kept)
    want, _ = moe.fused_moe_router(b["x"], rw, w["w1"], w["w2"], k, **flat)
    assert torch.equal(out, want)
    ids, _ = moe.moe_route(b["logits"], k)
    al = moe.moe_align(ids, E, 16)
    got = [moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU, b["x"], w["w1"], al, M, k, a_scale=b["x_scale"], w_scale=s)
           for s in (kept["w1_scale"], flat["w1_scale"])]
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    got = [moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN, got[0][0], w["w2"], al, M, k, a_scale=got[0][1], w_scale=s)[0]
           for s in (kept["w2_scale"], flat["w2_scale"])]
    assert torch.equal(got[0], got[1])
    host = [w["w1"].cpu(), w["w2"].cpu()]
    outs = []
    for kw in (kept, flat):
        cache = moe.ExpertCache(*host, E, w1_scale=kw["w1_scale"].cpu(), w2_scale=kw["w2_scale"].cpu())
        outs.append(cache(b["x"], b["logits"], k, x_scale=b["x_scale"]))
        torch.cuda.synchronize()
        cache.close()
    assert torch.equal(outs[0], outs[1])
