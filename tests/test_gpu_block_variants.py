"""The block-scaled e4m3 operators and the grouped router where their kernels
change shape: rings, splits, chunks, group layouts, large operands, skewed,
empty and poisoned batches, streams.  Bounds as in test_gpu_block_fp8 and
test_gpu_route_grouped.
"""
from functools import lru_cache

import pytest
import torch

import block_ref as ref
from test_gpu_block_fp8 import GROUPED, layer_ref, routed, within
from test_gpu_block_fp8 import weights as draw_weights
from test_gpu_route_grouped import check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


weights = lru_cache(maxsize=8)(draw_weights)


# ---------------------------------------------------------------- tile kernels

# (M, E, topk, H, I): many workgroups (shallow rings), several tiles an expert
# with more than eight weight tiles, the last group of them short
TILES = [(100, 64, 2, 1152, 640), (2100, 64, 2, 1152, 640), (700, 4, 2, 128, 1152), (90, 33, 1, 2176, 1152)]


@pytest.mark.parametrize("M,E,k,H,I", TILES)
@pytest.mark.parametrize("block_m", [32, 64, 128])
def test_gemm_tiles(dev, M, E, k, H, I, block_m):
    """Forty pairs of the batch against the float64 form."""
    import moe_layer_topk_amd as moe
    print(f"tiles M={M} E={E} k={k} H={H} I={I} block_m={block_m}", flush=True)
    ids = routed(M, E, k, M)
    P = M * k
    g = torch.Generator().manual_seed(M + H)
    x, xs = ref.quant(torch.randn(M, H, generator=g) * torch.exp(torch.randn(M, 1, generator=g)), 1)
    w1, s1 = weights(E, 2 * I, H, 1)
    w2, s2 = weights(E, H, I, 2)
    al = moe.moe_align(ids.to(dev), E, block_m)
    c, cs = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, x.to(dev), w1.to(dev), al, M, k, a_scale=xs.to(dev),
                                 w_scale=s1.to(dev))
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN_E4M3_ACT, c, w2.to(dev), al, M, k, a_scale=cs, w_scale=s2.to(dev))
    c, cs, y = c.cpu(), cs.cpu(), y.cpu().double()
    xv = ref.value(x, xs, 1)
    pairs = sorted({0, 1, P - 1, *torch.randint(0, P, (40,), generator=g).tolist()})
    for p in pairs:
        e = int(ids.reshape(-1)[p])
        one = torch.zeros(1, 1, dtype=torch.int32)
        act, bound = ref.silu_mul(*ref.products(xv[p // k:p // k + 1], ref.value(w1[e], s1[e], 128)[None], one, 1, True))
        blk = act.abs().view(I // 128, 128)
        top = blk.amax(1)
        got_s = cs[p].double()
        tol = bound.view(I // 128, 128).amax(1) / 448 + top / 448 * 2.0 ** -23
        within((got_s - top / 448).abs(), tol)
        a = ref.value(c[p:p + 1], cs[p:p + 1], 1)
        half = torch.maximum(act.abs() * 2.0 ** -4, got_s.repeat_interleave(128)[None] * 2.0 ** -10)
        within((a - act).abs(), half * (1 + 1e-6) + bound + tol.repeat_interleave(128)[None] * 448 * 1.01)
        yr, yb = ref.products(a, ref.value(w2[e], s2[e], 128)[None], one, 1, False)
        within((y[p:p + 1] - yr).abs(), yb + (yr.abs() + yb) * 2.0 ** -8)


@pytest.mark.parametrize("gate", [True, False])
def test_gemm_token_operand_past_4_gib(dev, gate):
    """Token rows past 4 GiB: every row is one of 1000, so every output row is
    that row's, bit for bit."""
    import moe_layer_topk_amd as moe
    M, E, K, N, base = 300_000, 3, 16384, 256, 1000
    assert M * K > 2 ** 32
    g = torch.Generator().manual_seed(5)
    x, xs = ref.quant(torch.randn(base, K, generator=g), 1)
    w, ws = weights(E, N, K, 6)
    x, xs, w, ws = x.view(torch.uint8).to(dev), xs.to(dev), w.to(dev), ws.to(dev)
    ids = (torch.arange(base, device=dev, dtype=torch.int32) % E).view(base, 1)
    row = torch.arange(M, device=dev) % base
    big, bigs = torch.empty(M, K, dtype=torch.uint8, device=dev), xs[row].contiguous()
    for i in range(0, M, base):
        big[i:i + base] = x
    kind = moe.MOE_GEMM_GATE_UP_SILU_E4M3 if gate else moe.MOE_GEMM_DOWN_E4M3_ACT
    for block_m in (32, 64, 128):
        print(f"far gate={gate} block_m={block_m}", flush=True)
        al = moe.moe_align(ids, E, block_m)
        want, wants = moe.moe_grouped_gemm(kind, x, w, al, base, 1, a_scale=xs, w_scale=ws)
        al = moe.moe_align(ids[row].contiguous(), E, block_m)
        got, gots = moe.moe_grouped_gemm(kind, big, w, al, M, 1, a_scale=bigs, w_scale=ws)
        torch.cuda.synchronize()
        bits = torch.uint8 if gate else torch.int16
        assert torch.equal(got.view(bits), want.view(bits)[row])
        if gate:
            assert torch.equal(gots, wants[row])


def test_gemm_same_expert_twice(dev):
    """A token that names one expert twice gets the same row twice."""
    import moe_layer_topk_amd as moe
    M, E, k, H, I = 40, 4, 3, 256, 256
    ids = routed(M, E, k, 1)
    ids[:, 2] = ids[:, 0]
    x, xs = ref.quant(torch.randn(M, H, generator=torch.Generator().manual_seed(1)), 1)
    w1, s1 = weights(E, 2 * I, H, 1)
    x, xs, w1, s1 = x.to(dev), xs.to(dev), w1.to(dev), s1.to(dev)
    for kind, block_m in ((moe.MOE_GEMM_GATE_UP_SILU, 16), (moe.MOE_GEMM_GATE_UP_SILU_E4M3, 32)):
        al = moe.moe_align(ids.to(dev), E, block_m)
        c, _ = moe.moe_grouped_gemm(kind, x, w1, al, M, k, a_scale=xs, w_scale=s1)
        c = c.view(torch.uint8).view(M, k, -1)
        assert torch.equal(c[:, 2], c[:, 0]) and not torch.equal(c[:, 1], c[:, 0])


# ----------------------------------------------------------------------- layer

def layer(M, E, k, H, I, dev, lg=None):
    g = torch.Generator().manual_seed(M + E + k)
    x = torch.randn(M, H, generator=g).bfloat16()
    lg = torch.randn(M, E, generator=g) if lg is None else lg
    w1, s1 = weights(E, 2 * I, H, 3)
    w2, s2 = weights(E, H, I, 4)
    return x, lg, (w1, s1, w2, s2), dict(w1=w1.to(dev), w2=w2.to(dev), w1_scale=s1.to(dev), w2_scale=s2.to(dev))


def close(out, want):
    assert float((out.cpu().double() - want).abs().max()) <= 3e-2 * float(want.abs().max())


# one token: every split of the down GEMM's units, more than one chunk of blocks
# a wavefront (topk 16 of 18 blocks; gate/up over 129)
@pytest.mark.parametrize("E,k,H,I", [(16, 1, 256, 384), (16, 2, 256, 384), (16, 3, 256, 384), (16, 5, 384, 128),
                                     (16, 9, 256, 384), (16, 16, 128, 2304), (2, 1, 16512, 128), (4, 2, 128, 8448)])
def test_layer_one_token(dev, E, k, H, I):
    import moe_layer_topk_amd as moe
    print(f"one token E={E} k={k} H={H} I={I}", flush=True)
    x, lg, w, d = layer(1, E, k, H, I, dev)
    out = moe.fused_moe(x.to(dev), lg.to(dev), topk=k, **d)
    want, _, _ = layer_ref(x, lg, k, *w)
    close(out, want)


# few rows and a long K: the down GEMM of a small batch in several splits
@pytest.mark.parametrize("M,E,k,H,I", [(2, 4, 1, 128, 4096), (4, 8, 2, 256, 1024), (16, 8, 2, 128, 2176), (3, 2, 2, 128, 1152)])
def test_layer_splits_its_down_gemm(dev, M, E, k, H, I):
    import moe_layer_topk_amd as moe
    print(f"splits M={M} E={E} k={k} H={H} I={I}", flush=True)
    x, lg, w, d = layer(M, E, k, H, I, dev)
    out = moe.fused_moe(x.to(dev), lg.to(dev), topk=k, **d)
    want, _, _ = layer_ref(x, lg, k, *w)
    close(out, want)
    assert torch.equal(out, moe.fused_moe(x.to(dev), lg.to(dev), topk=k, **d))


@pytest.mark.parametrize("M,E", [(20, 64), (64, 16), (300, 16)])
def test_layer_all_tokens_to_one_expert(dev, M, E):
    import moe_layer_topk_amd as moe
    lg = torch.randn(M, E, generator=torch.Generator().manual_seed(3))
    lg[:, 5] += 100.0
    x, lg, w, d = layer(M, E, 1, 256, 256, dev, lg)
    out = moe.fused_moe(x.to(dev), lg.to(dev), topk=1, **d)
    want, ids, _ = layer_ref(x, lg, 1, *w)
    assert bool((ids == 5).all())
    close(out, want)


# the grouped router inside the layer of a small batch: groups inside a lane,
# across lanes, of odd sizes, none; biased or not
@pytest.mark.parametrize("M", [1, 2, 7, 16, 17])
@pytest.mark.parametrize("E,G,T", [(256, 8, 4), (256, 2, 1), (256, 64, 8), (200, 5, 2), (40, 4, 3), (24, 1, 1)])
def test_layer_routes_as_the_router(dev, M, E, G, T):
    import moe_layer_topk_amd as moe
    k, H, I = 4, 128, 128
    g = torch.Generator().manual_seed(M + E)
    w1, s1 = (t.to(dev) for t in weights(E, 2 * I, H, 3))
    w2, s2 = (t.to(dev) for t in weights(E, H, I, 4))
    x = torch.randn(M, H, generator=g).bfloat16().to(dev)
    lg = torch.randn(M, E, generator=g)
    b = torch.randn(E, generator=g) * 0.05
    for score in ("softmax", "sigmoid"):
        for bias in (None, b):
            kw = dict(score=score, n_groups=G, topk_groups=T, group_top=2, scale=1.5)
            print(f"M={M} E={E} G={G} {score} bias={bias is not None}", flush=True)
            r = moe.Routing(bias=None if bias is None else bias.to(dev), **kw)
            ids = torch.empty(M, k, dtype=torch.int32, device=dev)
            wts = torch.empty(M, k, device=dev)
            moe.fused_moe_grouped(x, lg.to(dev), w1, w2, k, r, w1_scale=s1, w2_scale=s2, topk_ids=ids, topk_weights=wts)
            torch.cuda.synchronize()
            rid, rw = ref.route(lg, k, bias=bias, **kw)
            assert torch.equal(ids.cpu(), rid)
            assert bool(((wts.cpu().double() - rw).abs() <= 64 * 2.0 ** -24 * rw).all())


@pytest.mark.parametrize("M", [2, 20, 200])
def test_a_poisoned_token_stays_alone(dev, M):
    """NaN or an infinity in one token: its row is NaN, the others are as before."""
    import moe_layer_topk_amd as moe
    x, lg, _, d = layer(M, 8, 2, 256, 128, dev)
    lg = lg.to(dev)
    clean = moe.fused_moe(x.to(dev), lg, topk=2, **d)
    for v in (float("nan"), float("inf")):
        bad = x.clone()
        bad[1, 70] = v
        out = moe.fused_moe(bad.to(dev), lg, topk=2, **d)
        assert bool(torch.isnan(out[1]).all())
        keep = torch.arange(M) != 1
        assert torch.equal(out[keep.to(dev)], clean[keep.to(dev)])


@pytest.mark.parametrize("M", [1, 3, 40])
@pytest.mark.parametrize("slots", [4, 7])
def test_cached_layer_with_few_slots(dev, M, slots):
    """Experts that come and go through fewer slots than the layer has."""
    import moe_layer_topk_amd as moe
    E, k, H, I = 16, 2, 256, 128
    x, lg, (w1, s1, w2, s2), d = layer(M, E, k, H, I, dev)
    only = torch.zeros(E, dtype=torch.bool)
    cache = moe.ExpertCache(w1, w2, slots, w1_scale=s1, w2_scale=s2)
    for i in range(5):
        only[:] = True
        only[(torch.arange(4) + 3 * i) % E] = False  # four experts a batch
        l = lg.clone()
        l[:, only] -= 100.0
        out = cache(x.to(dev), l.to(dev), k)
        want = moe.fused_moe(x.to(dev), l.to(dev), topk=k, **d)
        close(out, want.cpu().double())
    cache.close()


@pytest.mark.parametrize("M", [1, 8, 200])
def test_layers_on_two_streams_at_once(dev, M):
    import moe_layer_topk_amd as moe
    x, lg, _, d = layer(M, 16, 4, 256, 256, dev)
    x, lg = x.to(dev), lg.to(dev)
    y = (x * 2).contiguous()
    want = [moe.fused_moe(t, lg, topk=4, **d) for t in (x, y)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.fused_moe((x, y)[i], lg, topk=4, **d))
    for s in streams:
        s.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_no_tokens(dev):
    import moe_layer_topk_amd as moe
    _, _, _, d = layer(1, 8, 2, 256, 128, dev)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=dev)
    lg = torch.empty(0, 8, device=dev)
    r = moe.Routing("sigmoid", n_groups=4, topk_groups=2)
    assert moe.fused_moe_grouped(x, lg, d["w1"], d["w2"], 2, r, w1_scale=d["w1_scale"], w2_scale=d["w2_scale"]).shape == (0, 256)
    assert moe.fused_moe(x, lg, topk=2, **d).shape == (0, 256)
    ids, wts = moe.moe_route_grouped(lg, 2, r)
    assert ids.shape == wts.shape == (0, 2)
    q, s = moe.moe_quant_block(x)
    assert q.shape == (0, 256) and s.shape == (0, 2)


def test_refusals_of_device_tensors(dev):
    """Strides, sizes and alignments that the kernels do not read are refused."""
    import moe_layer_topk_amd as moe
    M, E, k, H, I = 8, 8, 2, 256, 128
    x, lg, _, d = layer(M, E, k, H, I, dev)
    x, lg = x.to(dev), lg.to(dev)
    r = moe.Routing()
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_route_grouped(torch.randn(E, M, device=dev).t(), k, r)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_quant_block(torch.randn(H, M, device=dev).t())
    with pytest.raises(ValueError, match="contiguous"):
        moe.fused_moe(torch.randn(H, M, device=dev).bfloat16().t(), lg, topk=k, **d)
    with pytest.raises(ValueError, match="shape"):
        moe.fused_moe(x, lg, topk=k, **{**d, "w2_scale": d["w2_scale"][:, :, :0]})
    with pytest.raises(ValueError, match="bias"):
        moe.moe_route_grouped(lg, k, moe.Routing(bias=torch.zeros(E + 1, device=dev)))
    with pytest.raises(RuntimeError):  # rows that do not start on 16 bytes
        moe.moe_quant_block(torch.randn(M * H + 1, device=dev)[1:].view(M, H))
    q, qs = moe.moe_quant_block(x)
    al = moe.moe_align(torch.zeros(4, k, dtype=torch.int32, device=dev), E, 32)
    with pytest.raises(ValueError, match="align"):  # another batch's index system
        moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, q, d["w1"], al, M, k, a_scale=qs, w_scale=d["w1_scale"])
    with pytest.raises(ValueError, match="align"):  # of another number of experts
        al = moe.moe_align(torch.zeros(M, k, dtype=torch.int32, device=dev), E - 1, 32)
        moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, q, d["w1"], al, M, k, a_scale=qs, w_scale=d["w1_scale"])


# ---------------------------------------------------------------------- router

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
def test_route_wide_groups(dev, score, top):
    """Groups that span half the wavefront, and a third of the experts."""
    for M, E, G, T in ((50, 256, 2, 1), (50, 192, 3, 2), (50, 128, 2, 1), (50, 64, 2, 1), (50, 254, 2, 1)):
        print(f"wide M={M} E={E} G={G}", flush=True)
        lg, b = draw(M, E, E)
        check(dev, lg, 8, bias=b, score=score, n_groups=G, topk_groups=T, group_top=top)
        check(dev, lg, 8, score=score, n_groups=G, topk_groups=T, group_top=top)


def test_route_more_tokens_than_wavefronts(dev):
    lg, b = draw(20011, 16, 8)
    check(dev, lg, 4, bias=b, score="sigmoid", n_groups=4, topk_groups=2, group_top=2)


def test_route_replayed_from_a_graph(dev):
    import moe_layer_topk_amd as moe
    lg, b = draw(33, 128, 2)
    x = lg.to(dev)
    r = moe.Routing("sigmoid", b.to(dev), **{k: v for k, v in GROUPED.items() if k != "score"})
    ids, wts = moe.moe_route_grouped(x, 8, r)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        moe.moe_route_grouped(x, 8, r, topk_ids=ids, topk_weights=wts)
    for i in range(4):
        x.copy_(draw(33, 128, 20 + i)[0])
        ids.fill_(-1)
        gr.replay()
        torch.cuda.synchronize()
        got = ids.clone(), wts.clone()
        want = moe.moe_route_grouped(x, 8, r)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_quant_replayed_from_a_graph(dev):
    import moe_layer_topk_amd as moe
    x = torch.randn(130, 256, device=dev)
    for block_rows in (1, 128):
        q, s = moe.moe_quant_block(x, block_rows)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            moe.moe_quant_block(x, block_rows, q=q, scale=s)
        for i in range(4):
            x.copy_(torch.randn(130, 256, generator=torch.Generator().manual_seed(i)) * 10.0 ** i)
            q.view(torch.uint8).fill_(0)
            gr.replay()
            torch.cuda.synchronize()
            got = q.clone(), s.clone()
            wq, ws = moe.moe_quant_block(x, block_rows)
            assert torch.equal(got[0].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(got[1], ws)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_from_weights_quantised_on_the_device(dev, dtype):
    """moe_quant_block's blocks of 128 rows, stacked by expert, are the layer's weights."""
    import moe_layer_topk_amd as moe
    M, E, k, H, I = 24, 8, 2, 256, 384
    g = torch.Generator().manual_seed(4)
    w1 = (torch.randn(E, 2 * I, H, generator=g) * 0.05).to(dtype)
    w2 = (torch.randn(E, H, I, generator=g) * 0.05).to(dtype)
    x = torch.randn(M, H, generator=g).bfloat16()
    lg = torch.randn(M, E, generator=g)
    b = torch.randn(E, generator=g) * 0.05
    q1, s1 = (torch.stack(t) for t in zip(*(moe.moe_quant_block(w.to(dev), 128) for w in w1)))
    q2, s2 = (torch.stack(t) for t in zip(*(moe.moe_quant_block(w.to(dev), 128) for w in w2)))
    out = moe.fused_moe_grouped(x.to(dev), lg.to(dev), q1, q2, k, moe.Routing(bias=b.to(dev), **GROUPED), w1_scale=s1, w2_scale=s2)
    r1 = [torch.stack(t) for t in zip(*(ref.quant(w, 128) for w in w1))]
    r2 = [torch.stack(t) for t in zip(*(ref.quant(w, 128) for w in w2))]
    assert torch.equal(q1.cpu().view(torch.uint8), r1[0].view(torch.uint8)) and torch.equal(s2.cpu(), r2[1])
    want, _, _ = layer_ref(x, lg, k, *r1, *r2, bias=b, **GROUPED)
    close(out, want)
