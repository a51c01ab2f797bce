"""Block-scaled e4m3 on the GPU: the quantiser, the grouped GEMMs and the layer
against the float64 forms in block_ref.

Quantiser: codes and scales bit for bit (IEEE float32 quotients).
float32 act: within the bound of block_ref.products / silu_mul.
bfloat16 y: that bound plus half a bfloat16 step (2^-8) of the value.
e4m3 act: a code's value within half an e4m3 step (2^-4 of the value, 2^-10 of
the scale below the normals) of act, plus act's bound; scales within the bound
of the block's largest value / 448 plus two half-steps of 2^-24.
"""
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


def within(err, bound):
    """Every |error| within its bound; says how far the worst is."""
    worst = float((err / bound.clamp_min(1e-300)).max())
    assert worst <= 1.0, f"{worst} times the bound"


def same_codes(q, rq):
    assert torch.equal(q.cpu().view(torch.uint8), rq.view(torch.uint8))


# ------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 128), (1, 2048), (5, 4096), (127, 256), (128, 384), (129, 640), (300, 128)])
def test_quant(dev, dtype, block_rows, rows, K):
    import moe_layer_topk_amd as moe
    print(f"quant {dtype} block_rows={block_rows} rows={rows} K={K}", flush=True)
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3)).to(dtype)
    x[0, :128] = 0.0
    x[rows - 1, 1] = -0.0
    q, s = moe.moe_quant_block(x.to(dev), block_rows)
    rq, rs = ref.quant(x, block_rows)
    same_codes(q, rq)
    assert torch.equal(s.cpu(), rs)


@pytest.mark.parametrize("exp", [-149, -140, -126, -110, -90, -80, -60, 0, 60, 120])
def test_quant_magnitudes(dev, exp):
    """Blocks from the smallest subnormals to near the largest float32."""
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(exp + 200)
    x = (torch.randn(64, 256, generator=g).double() * 2.0 ** exp).float()
    q, s = moe.moe_quant_block(x.to(dev))
    rq, rs = ref.quant(x, 1)
    same_codes(q, rq)
    assert torch.equal(s.cpu(), rs)


def test_quant_ties(dev):
    """Quotients on and next to the borders between codes (amax 448: s = 1)."""
    import moe_layer_topk_amd as moe
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (codes[1:] + codes[:-1]) / 2
    up = torch.nextafter(mid, torch.tensor(1e9))
    dn = torch.nextafter(mid, torch.tensor(-1e9))
    v = torch.cat([mid, up, dn, -mid, -up, -dn])
    rows = torch.zeros(-(-v.numel() // 127), 128)
    rows[:, 0] = 448.0
    flat = torch.zeros(rows.shape[0] * 127)
    flat[:v.numel()] = v
    rows[:, 1:] = flat.view(-1, 127)
    for f in (1.0, 0.75, 3.0):
        x = rows * f
        q, s = moe.moe_quant_block(x.to(dev))
        rq, rs = ref.quant(x, 1)
        same_codes(q, rq)
        assert torch.equal(s.cpu(), rs)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_non_finite(dev, block_rows):
    import moe_layer_topk_amd as moe
    x = torch.randn(130, 384, generator=torch.Generator().manual_seed(1))
    x[3, 5] = float("inf")
    x[129, 200] = float("nan")
    x[64, 383] = float("-inf")
    q, s = moe.moe_quant_block(x.to(dev), block_rows)
    rq, rs = ref.quant(x, block_rows)
    same_codes(q, rq)
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(rs))
    assert torch.equal(torch.nan_to_num(s.cpu()), torch.nan_to_num(rs))


# ----------------------------------------------------------------------- GEMMs

def weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn)
    s = torch.empty(E, N // 128, K // 128)
    for e in range(E):
        # blocks of different size, so a wrong scale shows
        w = torch.randn(N, K, generator=g) * 0.05
        w *= torch.exp(torch.randn(N // 128, 1, K // 128, 1, generator=g)).expand(-1, 128, -1, 128).reshape(N, K)
        q[e], s[e] = ref.quant(w, 128)
    return q, s


def expert_values(q, s):
    return torch.stack([ref.value(q[e], s[e], 128) for e in range(q.shape[0])])


def routed(M, E, k, seed, only=None):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn(M, E, generator=g)
    if only is not None:
        lg[:, only:] -= 100.0
    return torch.topk(lg, k, dim=1).indices.to(torch.int32)


# (M, E, topk, H, I, experts the batch may use): one token to several tiles of
# an expert, tiles that end inside a row block, N an odd multiple of 128, K one
# block and an odd number of blocks
GEMMS = [(1, 4, 2, 128, 128, None), (3, 8, 2, 256, 128, None), (17, 4, 2, 384, 256, None), (40, 3, 1, 128, 384, 2),
         (70, 4, 3, 640, 128, None), (150, 2, 2, 256, 256, None), (9, 16, 8, 1152, 640, None), (33, 1, 1, 512, 384, None),
         (300, 5, 2, 128, 128, 3)]


@pytest.mark.parametrize("M,E,k,H,I,only", GEMMS)
@pytest.mark.parametrize("block_m", [32, 64, 128])
def test_gemm_e4m3_act(dev, M, E, k, H, I, only, block_m):
    import moe_layer_topk_amd as moe
    print(f"e4m3 act M={M} E={E} k={k} H={H} I={I} block_m={block_m}", flush=True)
    ids = routed(M, E, k, M, only)
    P = M * k
    g = torch.Generator().manual_seed(M + H)
    x, xs = ref.quant(torch.randn(M, H, generator=g) * torch.exp(torch.randn(M, 1, generator=g)), 1)
    w1, s1 = weights(E, 2 * I, H, 1)
    w2, s2 = weights(E, H, I, 2)
    al = moe.moe_align(ids.to(dev), E, block_m)
    c = torch.full((P + 1, I), 0x55, dtype=torch.uint8, device=dev)
    cs = torch.full((P + 1, I // 128), -3.0, device=dev)
    moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, x.to(dev), w1.to(dev), al, M, k, a_scale=xs.to(dev),
                         w_scale=s1.to(dev), c=c[:P], c_amax=cs[:P])
    torch.cuda.synchronize()
    assert bool((c[P] == 0x55).all()) and bool((cs[P] == -3.0).all())  # rows past the last pair stay
    act, bound = ref.silu_mul(*ref.products(ref.value(x, xs, 1), expert_values(w1, s1), ids, k, True))
    got_s = cs[:P].cpu().double()
    q = c[:P].cpu().view(torch.float8_e4m3fn)
    blk = act.abs().view(P, I // 128, 128)
    top, at = blk.max(2)
    tol = bound.view(P, I // 128, 128).amax(2) / 448 + top / 448 * 2.0 ** -23
    within((got_s - top / 448).abs(), tol)
    err = (ref.value(q, cs[:P].cpu(), 1) - act).abs()
    half = torch.maximum(act.abs() * 2.0 ** -4, got_s.repeat_interleave(128, 1) * 2.0 ** -10)
    within(err, half * (1 + 1e-6) + bound + tol.repeat_interleave(128, 1) * 448 * 1.01)
    # down on the kernel's own codes
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN_E4M3_ACT, c[:P], w2.to(dev), al, M, k, a_scale=cs[:P], w_scale=s2.to(dev))
    yr, yb = ref.products(ref.value(q, cs[:P].cpu(), 1), expert_values(w2, s2), ids, k, False)
    within((y.cpu().double() - yr).abs(), yb + (yr.abs() + yb) * 2.0 ** -8)


@pytest.mark.parametrize("M,E,k,H,I,only", GEMMS[:7])
@pytest.mark.parametrize("block_m", [1, 16, 64, 256])
def test_gemm_f32_act(dev, M, E, k, H, I, only, block_m):
    import moe_layer_topk_amd as moe
    print(f"f32 act M={M} E={E} k={k} H={H} I={I} block_m={block_m}", flush=True)
    ids = routed(M, E, k, M, only)
    P = M * k
    g = torch.Generator().manual_seed(M + H)
    x, xs = ref.quant(torch.randn(M, H, generator=g), 1)
    w1, s1 = weights(E, 2 * I, H, 1)
    w2, s2 = weights(E, H, I, 2)
    al = moe.moe_align(ids.to(dev), E, block_m)
    act, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU, x.to(dev), w1.to(dev), al, M, k, a_scale=xs.to(dev),
                                  w_scale=s1.to(dev))
    ar, ab = ref.silu_mul(*ref.products(ref.value(x, xs, 1), expert_values(w1, s1), ids, k, True))
    within((act.cpu().double() - ar).abs(), ab)
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN, act, w2.to(dev), al, M, k, w_scale=s2.to(dev))
    q, qs = ref.quant(act.cpu(), 1)  # the kernel quantises the float32 act it is given
    yr, yb = ref.products(ref.value(q, qs, 1), expert_values(w2, s2), ids, k, False)
    within((y.cpu().double() - yr).abs(), yb + (yr.abs() + yb) * 2.0 ** -8)


def test_gemm_skips_ids_out_of_range(dev):
    """Pairs routed to no expert keep their rows of c as they were."""
    import moe_layer_topk_amd as moe
    M, E, k, H, I = 20, 4, 2, 256, 128
    ids = routed(M, E, k, 1)
    ids[3, 1] = -1
    ids[7] = E
    x, xs = ref.quant(torch.randn(M, H, generator=torch.Generator().manual_seed(1)), 1)
    w1, s1 = weights(E, 2 * I, H, 1)
    al = moe.moe_align(ids.to(dev), E, 32)
    c = torch.full((M * k, I), 0x55, dtype=torch.uint8, device=dev)
    cs = torch.full((M * k, I // 128), -3.0, device=dev)
    moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, x.to(dev), w1.to(dev), al, M, k, a_scale=xs.to(dev),
                         w_scale=s1.to(dev), c=c, c_amax=cs)
    torch.cuda.synchronize()
    for p in (7, 14, 15):
        assert bool((c[p] == 0x55).all()) and float(cs[p, 0]) == -3.0
    assert bool((cs[[0, 1, 2, 8, 16]] > 0).all())


# ----------------------------------------------------------------------- layer

LAYERS = [(1, 16, 4, 256, 128), (1, 8, 2, 512, 384), (2, 16, 4, 256, 256), (16, 32, 8, 384, 128), (17, 8, 2, 256, 640),
          (90, 8, 2, 256, 128), (200, 8, 2, 384, 256), (500, 16, 4, 128, 128)]


def layer_ref(x, lg, k, w1, s1, w2, s2, **kw):
    ids, wts = ref.route(lg, k, **kw)
    q, qs = ref.quant(x, 1)
    act, _ = ref.silu_mul(*ref.products(ref.value(q, qs, 1), expert_values(w1, s1), ids, k, True))
    a, as_ = ref.quant(act.float(), 1)
    y, _ = ref.products(ref.value(a, as_, 1), expert_values(w2, s2), ids, k, False)
    return (y.view(x.shape[0], k, -1) * wts[:, :, None]).sum(1), ids, wts


GROUPED = dict(score="sigmoid", n_groups=4, topk_groups=2, group_top=2, renormalize=True, scale=2.5)


def layer_inputs(M, E, k, H, I, dev):
    g = torch.Generator().manual_seed(M + E)
    x = torch.randn(M, H, generator=g).bfloat16()
    lg = torch.randn(M, E, generator=g)
    b = torch.randn(E, generator=g) * 0.05
    w1, s1 = weights(E, 2 * I, H, 3)
    w2, s2 = weights(E, H, I, 4)
    return x, lg, b, (w1, s1, w2, s2), [t.to(dev) for t in (x, lg, w1, s1, w2, s2)]


@pytest.mark.parametrize("M,E,k,H,I", LAYERS)
def test_layer(dev, M, E, k, H, I):
    """fused_moe_grouped, fused_moe, fused_moe_noalloc and fused_moe_cached on
    block-scaled weights.  The intermediate's codes may differ by one where an
    act lies on a border to within float32's error, so the bar is the e4m3
    layer's (3e-2 of the largest output); the stages are held tighter above."""
    import moe_layer_topk_amd as moe
    print(f"layer M={M} E={E} k={k} H={H} I={I}", flush=True)
    x, lg, b, (w1, s1, w2, s2), (dx, dlg, dw1, ds1, dw2, ds2) = layer_inputs(M, E, k, H, I, dev)
    r = moe.Routing(bias=b.to(dev), **GROUPED)
    ids = torch.empty(M, k, dtype=torch.int32, device=dev)
    wts = torch.empty(M, k, device=dev)
    out = moe.fused_moe_grouped(dx, dlg, dw1, dw2, k, r, w1_scale=ds1, w2_scale=ds2, topk_ids=ids, topk_weights=wts)
    torch.cuda.synchronize()
    want, rid, rw = layer_ref(x, lg, k, w1, s1, w2, s2, bias=b, **GROUPED)
    assert torch.equal(ids.cpu(), rid)
    assert bool(((wts.cpu().double() - rw).abs() <= 64 * 2.0 ** -24 * rw).all())
    assert float((out.cpu().double() - want).abs().max()) <= 3e-2 * float(want.abs().max())
    again = moe.fused_moe_grouped(dx, dlg, dw1, dw2, k, r, w1_scale=ds1, w2_scale=ds2)
    assert torch.equal(again, out)  # the same bits every time
    soft = moe.fused_moe(dx, dlg, dw1, dw2, k, w1_scale=ds1, w2_scale=ds2)
    want, _, _ = layer_ref(x, lg, k, w1, s1, w2, s2)
    assert float((soft.cpu().double() - want).abs().max()) <= 3e-2 * float(want.abs().max())
    flat = moe.fused_moe_grouped(dx, dlg, dw1, dw2, k, moe.Routing(), w1_scale=ds1, w2_scale=ds2)
    assert float((flat.cpu().double() - want).abs().max()) <= 3e-2 * float(want.abs().max())
    noa = moe.fused_moe_noalloc(dx, dlg, dw1, dw2, k, w1_scale=ds1, w2_scale=ds2)
    assert torch.equal(noa, soft)
    cache = moe.ExpertCache(w1, w2, E, w1_scale=s1, w2_scale=s2)
    got = cache(dx, dlg, k)
    assert torch.equal(got, soft)
    cache.close()


@pytest.mark.parametrize("M", [16, 100, 300])
def test_layer_is_its_stages(dev, M):
    """The fused layer and the same steps through their own entry points: the
    same bits, except that a small batch keeps y in float32 where the stage
    rounds it to bfloat16 (half a step, 2^-8, of every weighted y, and half a
    step of the output, whose own rounding may fall the other way)."""
    import moe_layer_topk_amd as moe
    E, k, H, I = 16, 4, 384, 256
    x, lg, b, _, (dx, dlg, dw1, ds1, dw2, ds2) = layer_inputs(M, E, k, H, I, dev)
    r = moe.Routing(bias=b.to(dev), **GROUPED)
    out = moe.fused_moe_grouped(dx, dlg, dw1, dw2, k, r, w1_scale=ds1, w2_scale=ds2)
    ids, wts = moe.moe_route_grouped(dlg, k, r)
    al = moe.moe_align(ids, E, moe.moe_block_m(moe.MOE_FP8_BLOCK, M, E, k))
    q, qs = moe.moe_quant_block(dx)
    a, as_ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, q, dw1, al, M, k, a_scale=qs, w_scale=ds1)
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN_E4M3_ACT, a, dw2, al, M, k, a_scale=as_, w_scale=ds2)
    want = moe.moe_combine(y, wts, k)
    if M >= 100:
        assert torch.equal(out, want)
    half = (y.float().abs().view(M, k, H) * wts[:, :, None]).sum(1).double() * 2.0 ** -8
    within((out.double() - want.double()).abs().cpu(), (half + (want.double().abs() + half) * 2.0 ** -7).cpu())


@pytest.mark.parametrize("name", ["f32", "bf16", "fp8", "w4a16"])
@pytest.mark.parametrize("M", [1, 20, 200])
def test_grouped_router_on_every_dtype(dev, name, M):
    """fused_moe_grouped with the plain softmax router is fused_moe; with a
    grouped one its ids and weights are moe_route_grouped's."""
    from dataclasses import replace

    import moe_layer_topk_amd as moe
    from workloads import CONFIGS, layer_batch, layer_weights
    base = {"f32": "tiny_f32", "bf16": "finegrained_bf16", "fp8": "fp8_e4m3", "w4a16": "finegrained_w4a16"}[name]
    cfg = replace(CONFIGS[base], E=16, topk=4, H=512, I=256, router="normal")
    w = layer_weights(cfg, dev)
    bt = layer_batch(cfg, M, dev)
    kw = dict(x_scale=bt["x_scale"], w1_scale=w["w1_scale"], w2_scale=w["w2_scale"])
    plain = moe.fused_moe(bt["x"], bt["logits"], w["w1"], w["w2"], 4, **kw)
    same = moe.fused_moe_grouped(bt["x"], bt["logits"], w["w1"], w["w2"], 4, moe.Routing(), **kw)
    tol = 3e-2 if name == "fp8" else 1e-2
    assert float((plain.float() - same.float()).abs().max()) <= tol * float(plain.float().abs().max())
    b = torch.randn(16, generator=torch.Generator().manual_seed(2)).to(dev) * 0.05
    r = moe.Routing(bias=b, **GROUPED)
    ids = torch.empty(M, 4, dtype=torch.int32, device=dev)
    wts = torch.empty(M, 4, device=dev)
    moe.fused_moe_grouped(bt["x"], bt["logits"], w["w1"], w["w2"], 4, r, topk_ids=ids, topk_weights=wts, **kw)
    rid, rw = moe.moe_route_grouped(bt["logits"], 4, r)
    assert torch.equal(ids, rid) and torch.equal(wts, rw)


def test_layer_from_hidden_states(dev):
    import moe_layer_topk_amd as moe
    for M in (1, 8, 40):
        x, _, _, (w1, s1, w2, s2), (dx, _, dw1, ds1, dw2, ds2) = layer_inputs(M, 8, 2, 256, 128, dev)
        rw = torch.randn(8, 256, generator=torch.Generator().manual_seed(7)) * 0.1
        out, lg = moe.fused_moe_router(dx, rw.to(dev), dw1, dw2, 2, w1_scale=ds1, w2_scale=ds2)
        want, _, _ = layer_ref(x, lg.cpu(), 2, w1, s1, w2, s2)
        assert float((lg.cpu().double() - x.double() @ rw.double().t()).abs().max()) <= 1e-4
        assert float((out.cpu().double() - want).abs().max()) <= 3e-2 * float(want.abs().max())


def test_layer_replayed_from_a_graph(dev):
    """Captured once, replayed with new inputs and the program's own work between."""
    import moe_layer_topk_amd as moe
    for M in (1, 24, 200):
        E, k, H, I = 16, 4, 256, 256
        _, lg, b, _, (dx, dlg, dw1, ds1, dw2, ds2) = layer_inputs(M, E, k, H, I, dev)
        r = moe.Routing(bias=b.to(dev), **GROUPED)
        ws = torch.empty(moe.fused_moe_workspace_size(moe.MOE_FP8_BLOCK, M, E, k, H, I), dtype=torch.uint8, device=dev)
        out = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
        call = lambda: moe.fused_moe_grouped(dx, dlg, dw1, dw2, k, r, w1_scale=ds1, w2_scale=ds2, workspace=ws, out=out)  # noqa: E731
        call()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        for i in range(4):
            g = torch.Generator().manual_seed(100 + i)
            dx.copy_(torch.randn(M, H, generator=g).bfloat16())
            dlg.copy_(torch.randn(M, E, generator=g))
            ws.fill_(0xA5)
            gr.replay()
            torch.cuda.synchronize()
            got = out.clone()
            out.zero_()
            call()
            assert torch.equal(got, out)
