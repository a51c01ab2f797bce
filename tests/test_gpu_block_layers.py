"""Small batches of block-scaled layers with wide experts, which pass the
intermediate as e4m3 codes (32 blocks of columns and more for 16 experts: more
than 512 tile workgroups), and the routers inside a layer's launches on rows
that are masked, poisoned or too close for float32.  Bounds as in
test_gpu_block_fp8 and test_gpu_route_grouped.
"""
import math
from functools import lru_cache

import pytest
import torch

import block_ref as ref
from test_gpu_block_fp8 import GROUPED, layer_ref
from test_gpu_block_fp8 import weights as draw_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


weights = lru_cache(maxsize=4)(draw_weights)


def wide(M, E, k, H, I, dev):
    g = torch.Generator().manual_seed(M + E)
    x = torch.randn(M, H, generator=g).bfloat16()
    lg = torch.randn(M, E, generator=g)
    w1, s1 = weights(E, 2 * I, H, 3)
    w2, s2 = weights(E, H, I, 4)
    return x, lg, (w1, s1, w2, s2), dict(w1=w1.to(dev), w2=w2.to(dev), w1_scale=s1.to(dev), w2_scale=s2.to(dev))


# (M, E, topk, H, I): every one with at most 8 rows an expert
WIDE = [(1, 32, 16, 128, 4224), (2, 32, 16, 128, 4224), (16, 32, 16, 128, 4224), (17, 64, 12, 128, 2176), (3, 24, 12, 256, 4224)]


@pytest.mark.parametrize("M,E,k,H,I", WIDE)
def test_wide_experts(dev, M, E, k, H, I):
    """The layer against the float64 form, and its steps through their own entry
    points, the kinds on e4m3 act: the same bits."""
    import moe_layer_topk_amd as moe
    print(f"wide M={M} E={E} k={k} H={H} I={I}", flush=True)
    x, lg, w, d = wide(M, E, k, H, I, dev)
    dx, dlg = x.to(dev), lg.to(dev)
    b = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.05
    r = moe.Routing(bias=b.to(dev), **GROUPED)
    ids = torch.empty(M, k, dtype=torch.int32, device=dev)
    wts = torch.empty(M, k, device=dev)
    out = moe.fused_moe_grouped(dx, dlg, topk=k, routing=r, topk_ids=ids, topk_weights=wts, **d)
    torch.cuda.synchronize()
    want, rid, rw = layer_ref(x, lg, k, *w, bias=b, **GROUPED)
    assert torch.equal(ids.cpu(), rid)
    assert bool(((wts.cpu().double() - rw).abs() <= 64 * 2.0 ** -24 * rw).all())
    assert float((out.cpu().double() - want).abs().max()) <= 3e-2 * float(want.abs().max())
    al = moe.moe_align(ids, E, moe.moe_block_m(moe.MOE_FP8_BLOCK, M, E, k))
    q, qs = moe.moe_quant_block(dx)
    a, as_ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, q, d["w1"], al, M, k, a_scale=qs, w_scale=d["w1_scale"])
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN_E4M3_ACT, a, d["w2"], al, M, k, a_scale=as_, w_scale=d["w2_scale"])
    assert torch.equal(moe.moe_combine(y, wts, k), out)


@pytest.mark.parametrize("M,E,k,H,I", WIDE[:4])
def test_wide_experts_through_every_entry_point(dev, M, E, k, H, I):
    import moe_layer_topk_amd as moe
    print(f"wide M={M} E={E} k={k} H={H} I={I}", flush=True)
    x, lg, (w1, s1, w2, s2), d = wide(M, E, k, H, I, dev)
    dx, dlg = x.to(dev), lg.to(dev)
    soft = moe.fused_moe(dx, dlg, topk=k, **d)
    assert torch.equal(moe.fused_moe_noalloc(dx, dlg, topk=k, **d), soft)
    assert torch.equal(moe.fused_moe_grouped(dx, dlg, topk=k, routing=moe.Routing(), **d), soft)
    cache = moe.ExpertCache(w1, w2, E, w1_scale=s1, w2_scale=s2)
    for _ in range(2):  # every expert copied, then found
        assert torch.equal(cache(dx, dlg, k), soft)
    cache.close()
    rw = torch.randn(E, H, generator=torch.Generator().manual_seed(7)).to(dev) * 0.1
    out, scores = moe.fused_moe_router(dx, rw, topk=k, **d)
    assert torch.equal(moe.fused_moe(dx, scores, topk=k, **d), out)


def test_wide_experts_replayed_from_a_graph(dev):
    import moe_layer_topk_amd as moe
    M, E, k, H, I = WIDE[1]
    x, lg, _, d = wide(M, E, k, H, I, dev)
    dx, dlg = x.to(dev), lg.to(dev)
    ws = torch.empty(moe.fused_moe_workspace_size(moe.MOE_FP8_BLOCK, M, E, k, H, I), dtype=torch.uint8, device=dev)
    out = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    call = lambda: moe.fused_moe(dx, dlg, topk=k, workspace=ws, out=out, **d)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        g = torch.Generator().manual_seed(100 + i)
        dx.copy_(torch.randn(M, H, generator=g).bfloat16())
        dlg.copy_(torch.randn(M, E, generator=g))
        ws.fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        call()
        assert torch.equal(got, out)


def hard_rows():
    """Logits [12, 64]: infinities, NaN, masked rows and groups, near ties."""
    inf, nan = math.inf, math.nan
    g = torch.Generator().manual_seed(5)
    lg = torch.randn(12, 64, generator=g)
    lg[0] = -inf
    lg[1, 3:] = -inf
    lg[2, 5] = nan
    lg[3] = nan
    lg[4, 7] = inf
    lg[5, [9, 50]] = inf
    lg[6] = torch.finfo(torch.float32).min
    lg[7, ::2] = torch.finfo(torch.float32).min
    lg[8, 1:] = -200.0
    lg[9, :32] = -inf
    for t in (10, 11):
        lg[t, 1::2] = torch.nextafter(lg[t, 0::2], torch.full((32,), inf if t % 2 else -inf))
    return lg, torch.randn(64, generator=g) * 0.05


# (V = 4 experts a lane here: 8 groups are two lanes each, 2 of 32 eight, 64 of 1 a part of one)
@pytest.mark.parametrize("M", [1, 12])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,T,top", [(1, 1, 1), (8, 3, 2), (2, 1, 1), (64, 20, 1)])
@pytest.mark.parametrize("bias", ["none", "small", "zero", "poisoned"])
def test_layer_routes_hard_rows(dev, M, score, G, T, top, bias):
    import moe_layer_topk_amd as moe
    E, k, H, I = 64, 8, 128, 128
    lg, b = hard_rows()
    if bias == "zero":
        b = torch.zeros(E)
    if bias == "poisoned":
        b[4], b[5], b[6] = math.inf, -math.inf, math.nan
    b = None if bias == "none" else b
    kw = dict(score=score, n_groups=G, topk_groups=T, group_top=top, scale=1.5)
    w1, s1 = (t.to(dev) for t in weights(E, 2 * I, H, 3))
    w2, s2 = (t.to(dev) for t in weights(E, H, I, 4))
    x = torch.randn(M, H, generator=torch.Generator().manual_seed(M)).bfloat16().to(dev)
    r = moe.Routing(bias=None if b is None else b.to(dev), **kw)
    rid, rw = ref.route(lg, k, bias=b, **kw)
    for t in range(0, 12, M):
        part = slice(t, t + M)
        ids = torch.empty(M, k, dtype=torch.int32, device=dev)
        wts = torch.empty(M, k, device=dev)
        moe.fused_moe_grouped(x, lg[part].to(dev), w1, w2, k, r, w1_scale=s1, w2_scale=s2, topk_ids=ids, topk_weights=wts)
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu(), rid[part]), t
        # (span of a row's finite logits, at most 104)
        assert bool(((wts.cpu().double() - rw[part]).abs() <= (32 + 104) * 2.0 ** -24 * rw[part] + 2.0 ** -150).all()), t
