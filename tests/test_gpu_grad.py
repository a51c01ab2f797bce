"""The experts' products as a training step needs them (gate and up before
SiLU-and-mul, gradients of rows and weights) against float64.

Bounds: a float32 sum of n products of bfloat16 values (exact in float32) is off by
at most n U times the sum of the products' magnitudes, in whatever order; twice
that for a matrix instruction that keeps a bit less.  The outputs add their own
rounding.  Through SiLU-and-mul the float32 factors add 16 U, their exponential
and quotient included."""
import pytest
import torch

import train_ref as ref
from train_ref import HALF, U, close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


def routes(M, k, E, how, seed=0):
    """ids [M, k]: spread, all to one expert, or with ids that are no expert."""
    g = torch.Generator().manual_seed(100 + seed)
    if how == "one":
        return torch.full((M, k), E - 1, dtype=torch.int32)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    if how == "dropped":
        ids = torch.where(torch.rand(M, k, generator=g) < 0.3, torch.where(torch.rand(M, k, generator=g) < 0.5, -1, E), ids).int()
    return ids


def randn(g, *shape, size=1.0):
    return (torch.randn(*shape, generator=g) * size).to(BF)


def pairs_of(ids, E):
    flat = ids.reshape(-1)
    return [(flat == e).nonzero().flatten() for e in range(E)]


#        M    k  E   H    I   block_m how
CASES = [(1, 1, 1, 128, 128, 64, "spread"),
         (1, 8, 16, 256, 128, 64, "spread"),
         (5, 2, 4, 384, 256, 128, "spread"),
         (63, 4, 8, 640, 384, 64, "spread"),
         (130, 2, 3, 256, 640, 128, "dropped"),
         (200, 3, 7, 128, 128, 64, "one"),
         (65, 1, 2, 512, 896, 128, "one"),
         (97, 6, 40, 256, 256, 128, "dropped"),
         (300, 2, 2, 1152, 128, 64, "spread")]


def setup(dev, M, k, E, H, I, block_m, how, seed):
    import moe_layer_topk_amd as moe
    ids = routes(M, k, E, how, seed)
    al = moe.moe_align(ids.to(dev), E, block_m)
    return ids, pairs_of(ids, E), al, torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("M,k,E,H,I,block_m,how", CASES)
def test_gate_up(dev, M, k, E, H, I, block_m, how):
    import moe_layer_topk_amd as moe
    ids, pairs, al, g = setup(dev, M, k, E, H, I, block_m, how, 1)
    x, w = randn(g, M, H), randn(g, E, 2 * I, H, size=0.05)
    z = torch.full((M * k, 2 * I), 7.0, dtype=BF, device=dev)
    moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x.to(dev), w.to(dev), al, M, k, c=z)
    want, bound = torch.full((M * k, 2 * I), 7.0, dtype=torch.float64), torch.zeros(M * k, 2 * I, dtype=torch.float64)
    for e, p in enumerate(pairs):
        a, b = x[p // k].double(), w[e].double()
        want[p] = a @ b.t()
        bound[p] = HALF[BF] * want[p].abs() + 2 * H * U * (a.abs() @ b.abs().t())
    close(z, want, bound, "z")  # rows of pairs without an expert as they were


@pytest.mark.parametrize("M,k,E,H,I,block_m,how", CASES)
def test_dx_plain(dev, M, k, E, H, I, block_m, how):
    import moe_layer_topk_amd as moe
    ids, pairs, al, g = setup(dev, M, k, E, H, I, block_m, how, 2)
    for kind, N, K in ((moe.MOE_GEMM_GATE_UP, 2 * I, H), (moe.MOE_GEMM_DOWN, H, I)):
        dc, w = randn(g, M * k, N), randn(g, E, N, K, size=0.05)
        held = torch.cat(pairs)
        lost = torch.ones(M * k, dtype=torch.bool)
        lost[held] = False
        dc[lost] = float("nan")  # rows of no expert are read into nothing
        da = torch.full((M * k, K), 7.0, dtype=BF, device=dev)
        got, act = moe.moe_grouped_gemm_dx(kind, dc.to(dev), w.to(dev), al, M, k, da=da)
        assert got is da and act is None
        want, bound = torch.full((M * k, K), 7.0, dtype=torch.float64), torch.zeros(M * k, K, dtype=torch.float64)
        for e, p in enumerate(pairs):
            a, b = dc[p].double(), w[e].double()
            want[p] = a @ b
            bound[p] = HALF[BF] * want[p].abs() + 2 * N * U * (a.abs() @ b.abs())
        close(da, want, bound, f"da {N}x{K}")


def silu_grad(d, z):
    """(dz, act, magnitudes of dz per unit of error in d)"""
    I = z.shape[1] // 2
    gt, up = z[:, :I], z[:, I:]
    s = torch.sigmoid(gt)
    slope = up * s * (1 + gt * (1 - s))
    mag = up.abs() * s * (1 + gt.abs() * (1 - s))
    return (torch.cat([d * slope, d * gt * s], 1), gt * s * up, torch.cat([slope.abs(), (gt * s).abs()], 1),
            torch.cat([d.abs() * mag, (d * gt * s).abs()], 1))


@pytest.mark.parametrize("M,k,E,H,I,block_m,how", CASES)
def test_dx_through_silu(dev, M, k, E, H, I, block_m, how):
    import moe_layer_topk_amd as moe
    ids, pairs, al, g = setup(dev, M, k, E, H, I, block_m, how, 3)
    dy, w, z = randn(g, M * k, H), randn(g, E, H, I, size=0.05), randn(g, M * k, 2 * I, size=3.0)
    z[0, 0], z[0, I] = -80.0, 3.0   # far sides of the sigmoid
    z[-1, 1], z[-1, I + 1] = 80.0, -3.0
    da = torch.full((M * k, 2 * I), 7.0, dtype=BF, device=dev)
    act = torch.full((M * k, I), 7.0, dtype=BF, device=dev)
    moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy.to(dev), w.to(dev), al, M, k, z=z.to(dev), da=da, act=act)
    want, bound = torch.full((M * k, 2 * I), 7.0, dtype=torch.float64), torch.zeros(M * k, 2 * I, dtype=torch.float64)
    wact, bact = torch.full((M * k, I), 7.0, dtype=torch.float64), torch.zeros(M * k, I, dtype=torch.float64)
    for e, p in enumerate(pairs):
        a, b = dy[p].double(), w[e].double()
        d, e_d = a @ b, 2 * H * U * (a.abs() @ b.abs())
        want[p], wact[p], slope, mag = silu_grad(d, z[p].double())
        bound[p] = HALF[BF] * want[p].abs() + torch.cat([e_d, e_d], 1) * slope * 1.01 + 16 * U * mag + 1e-38
        bact[p] = (HALF[BF] + 16 * U) * wact[p].abs() + 1e-38
    close(da, want, bound, "dz")
    close(act, wact, bact, "act")


@pytest.mark.parametrize("block_m", [64, 128])
def test_dx_through_silu_of_many_rows(dev, block_m):
    """Over 96 MB of z, gradients and activations: they pass the caches."""
    import moe_layer_topk_amd as moe
    M, k, E, H, I = 4001, 2, 5, 128, 1408
    ids, pairs, al, g = setup(dev, M, k, E, H, I, block_m, "dropped", 9)
    dy, w, z = randn(g, M * k, H), randn(g, E, H, I, size=0.05), randn(g, M * k, 2 * I, size=3.0)
    da, act = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy.to(dev), w.to(dev), al, M, k, z=z.to(dev),
                                      da=torch.full((M * k, 2 * I), 7.0, dtype=BF, device=dev),
                                      act=torch.full((M * k, I), 7.0, dtype=BF, device=dev))
    for e, p in enumerate(pairs):
        p = p[::37]
        a, b = dy[p].double(), w[e].double()
        d, e_d = a @ b, 2 * H * U * (a.abs() @ b.abs())
        want, wact, slope, mag = silu_grad(d, z[p].double())
        close(da[p.to(dev)], want, HALF[BF] * want.abs() + torch.cat([e_d, e_d], 1) * slope * 1.01 + 16 * U * mag + 1e-38, "dz")
        close(act[p.to(dev)], wact, (HALF[BF] + 16 * U) * wact.abs() + 1e-38, "act")
    lost = torch.ones(M * k, dtype=torch.bool)
    lost[torch.cat(pairs)] = False
    assert (da[lost.to(dev)] == 7.0).all() and (act[lost.to(dev)] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,k,E,H,I,block_m,how", CASES + [(5000, 1, 1, 128, 128, 16, "one"), (4097, 2, 2, 128, 384, 1, "spread"),
                                                           (40, 2, 9, 256, 128, 256, "one")])
def test_dw(dev, M, k, E, H, I, block_m, how, dtype):
    import moe_layer_topk_amd as moe
    ids, pairs, al, g = setup(dev, M, k, E, H, I, block_m, how, 4)
    P = M * k
    lost = torch.ones(P, dtype=torch.bool)
    lost[torch.cat(pairs)] = False
    for kind, N, K, rows in ((moe.MOE_GEMM_GATE_UP, 2 * I, H, M), (moe.MOE_GEMM_DOWN, H, I, P)):
        dc, a = randn(g, P, N), randn(g, rows, K)
        dc[lost] = float("nan")
        if kind == moe.MOE_GEMM_DOWN:
            a[lost] = float("inf")
        dw = moe.moe_grouped_gemm_dw(kind, dc.to(dev), a.to(dev), al, M, k, dtype=dtype,
                                     dw=torch.full((E, N, K), float("nan"), dtype=dtype, device=dev))
        for e, p in enumerate(pairs):
            d, v = dc[p].double(), a[p // k if kind == moe.MOE_GEMM_GATE_UP else p].double()
            want = d.t() @ v
            bound = HALF[dtype] * want.abs() + 2 * max(len(p), 1) * U * (d.abs().t() @ v.abs())
            close(dw[e], want, bound, f"dw expert {e} {N}x{K}")


def test_adjoint(dev):
    """<dc, W a> = <W^T dc, a> = <dW, W>: the three calls agree with each other and with
    differences (the product is linear in each operand).  Each bfloat16 result is off
    by 2^-8 of itself, alternating in sign: 2^-8 times the norms bounds their sums."""
    import moe_layer_topk_amd as moe
    M, k, E, H, I = 150, 2, 4, 256, 384
    ids, pairs, al, g = setup(dev, M, k, E, H, I, 64, "spread", 5)
    x, w, dz = randn(g, M, H).to(dev), randn(g, E, 2 * I, H, size=0.05).to(dev), randn(g, M * k, 2 * I).to(dev)
    z = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, w, al, M, k)[0]
    da, _ = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_GATE_UP, dz, w, al, M, k)
    dw = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_GATE_UP, dz, x, al, M, k, dtype=F32)
    a = x.repeat_interleave(k, 0)

    def dot(u, v):
        return float((u.double() * v.double()).sum()), 2.0 ** -8 * float(u.double().norm() * v.double().norm())

    (s0, b0), (s1, b1), (s2, _) = dot(z, dz), dot(da, a), dot(dw, w)
    assert abs(s0 - s2) <= b0 and abs(s1 - s2) <= b1, (s0, s1, s2, b0, b1)
    v = randn(g, M, H).to(dev)  # a difference in x
    zp = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, (x + v).to(BF), w, al, M, k)[0]
    step = ((x + v).to(BF).double() - x.double())
    dx, _ = moe.moe_permute_backward(da, topk=k)
    assert abs(dot(zp, dz)[0] - s0 - dot(step, dx)[0]) <= b0 + dot(zp, dz)[1] + dot(step, dx)[1]


def test_gate_up_matches_the_fused_kind(dev):
    """SiLU-and-mul of z is the fused kind's act but for z's rounding (2^-8 of gate and up
    each, the slope of silu at most 1.1: 3 roundings of the sizes involved)."""
    import moe_layer_topk_amd as moe
    M, k, E, H, I = 200, 2, 4, 256, 256
    ids, pairs, al, g = setup(dev, M, k, E, H, I, 64, "spread", 6)
    x, w = randn(g, M, H).to(dev), randn(g, E, 2 * I, H, size=0.05).to(dev)
    z = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, w, al, M, k)[0].double().cpu()
    act = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU, x, w, al, M, k)[0]
    gt, up = z[:, :I], z[:, I:]
    close(act, ref.silu_mul(z), 2.0 ** -8 * 1.1 * (3 * gt.abs() * up.abs()) + 1e-6, "act")


def test_empty_batch(dev):
    import moe_layer_topk_amd as moe
    ids = torch.empty(0, 2, dtype=torch.int32, device=dev)
    al = moe.moe_align(ids, 4, 64)
    z = torch.empty(0, 256, dtype=BF, device=dev)
    x = torch.empty(0, 128, dtype=BF, device=dev)
    w = torch.zeros(4, 256, 128, dtype=BF, device=dev)
    assert moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, w, al, 0, 2)[0].shape == (0, 256)
    assert moe.moe_grouped_gemm_dx(moe.MOE_GEMM_GATE_UP, z, w, al, 0, 2)[0].shape == (0, 128)
    for dt in (BF, F32):
        dw = torch.full((4, 256, 128), 7.0, dtype=dt, device=dev)
        moe.moe_grouped_gemm_dw(moe.MOE_GEMM_GATE_UP, z, x, al, 0, 2, dw=dw)
        assert not dw.any()


def test_operands_past_four_gib(dev):
    """dc of 70000 x 32768 (4.6 GB): rows and columns from its far end."""
    import moe_layer_topk_amd as moe
    M, N, K = 70000, 32768, 128
    ids = torch.zeros(M, 1, dtype=torch.int32, device=dev)
    al = moe.moe_align(ids, 1, 128)
    g = torch.Generator(device=dev).manual_seed(7)
    dc = torch.empty(M, N, dtype=BF, device=dev)
    for i in range(0, M, 10000):
        dc[i:i + 10000] = torch.randn(10000, N, generator=g, device=dev).to(BF)
    w = (torch.randn(1, N, K, generator=g, device=dev) * 0.02).to(BF)
    a = torch.randn(M, K, generator=g, device=dev).to(BF)
    da, _ = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dc, w, al, M, 1)
    for r in (slice(0, 3), slice(33333, 33336), slice(M - 3, M)):
        d, v = dc[r].double(), w[0].double()
        want = d @ v
        close(da[r], want.cpu(), (HALF[BF] * want.abs() + 2 * N * U * (d.abs() @ v.abs())).cpu(), "da")
    w1 = (torch.randn(1, 256, N, generator=g, device=dev) * 0.02).to(BF)
    z, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, dc, w1, al, M, 1)  # (dc as the tokens)
    for r in (slice(0, 3), slice(M - 3, M)):
        d, v = dc[r].double(), w1[0].double().t()
        want = d @ v
        close(z[r], want.cpu(), (HALF[BF] * want.abs() + 2 * N * U * (d.abs() @ v.abs())).cpu(), "z")
    dw = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_DOWN, dc, a, al, M, 1, dtype=F32)
    for c in (slice(0, 3), slice(N - 3, N)):
        d, v = dc[:, c].double(), a.double()
        want = d.t() @ v
        close(dw[0, c], want.cpu(), (HALF[F32] * want.abs() + 2 * M * U * (d.abs().t() @ v.abs())).cpu(), "dw")


def test_repeat_streams_and_graphs(dev):
    """The same bits every time, on another stream and in a replayed graph."""
    import moe_layer_topk_amd as moe
    M, k, E, H, I = 300, 4, 8, 512, 384
    ids, pairs, al, g = setup(dev, M, k, E, H, I, 64, "spread", 8)
    x, w1, w2 = randn(g, M, H).to(dev), randn(g, E, 2 * I, H, size=0.05).to(dev), randn(g, E, H, I, size=0.05).to(dev)
    dy = randn(g, M * k, H).to(dev)
    z, dz = torch.empty(M * k, 2 * I, dtype=BF, device=dev), torch.empty(M * k, 2 * I, dtype=BF, device=dev)
    act, da = torch.empty(M * k, I, dtype=BF, device=dev), torch.empty(M * k, H, dtype=BF, device=dev)
    dw1, dw2 = torch.empty(E, 2 * I, H, device=dev), torch.empty(E, H, I, dtype=BF, device=dev)
    outs = (z, dz, act, da, dw1, dw2)

    def step():
        moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, w1, al, M, k, c=z)
        moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy, w2, al, M, k, z=z, da=dz, act=act)
        moe.moe_grouped_gemm_dw(moe.MOE_GEMM_DOWN, dy, act, al, M, k, dw=dw2)
        moe.moe_grouped_gemm_dx(moe.MOE_GEMM_GATE_UP, dz, w1, al, M, k, da=da)
        moe.moe_grouped_gemm_dw(moe.MOE_GEMM_GATE_UP, dz, x, al, M, k, dw=dw1)

    def run(f):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        f()
        torch.cuda.synchronize()
        return [t.clone() for t in outs]

    first = run(step)
    assert all(torch.equal(a, b) for a, b in zip(first, run(step)))
    side = torch.cuda.Stream(dev)

    def on_side():
        with torch.cuda.stream(side):
            step()

    assert all(torch.equal(a, b) for a, b in zip(first, run(on_side)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(randn(g, M, H).to(dev))
        got = run(graph.replay)
        assert all(torch.equal(a, b) for a, b in zip(got, run(step)))


#       M    k  E    H     I    block_m how: sizes of many workgroups, for experts of few rows and of many
MANY = [(120, 2, 160, 256, 256, 64, "spread"),
        (121, 2, 160, 384, 384, 128, "dropped"),
        (1030, 2, 20, 1152, 1152, 64, "spread"),
        (1030, 2, 20, 1152, 1152, 128, "dropped"),
        (1000, 2, 4, 1280, 1280, 128, "one")]


@pytest.mark.parametrize("M,k,E,H,I,block_m,how", MANY)
def test_products_of_many_workgroups(dev, M, k, E, H, I, block_m, how):
    test_gate_up(dev, M, k, E, H, I, block_m, how)
    test_dx_plain(dev, M, k, E, H, I, block_m, how)
    test_dx_through_silu(dev, M, k, E, H, I, block_m, how)


@pytest.mark.parametrize("M,k,E,H,I,block_m,how", [(3, 1, 2, 128, 2176, 64, "spread"),    # sums of one stage and of many
                                                   (65, 1, 1, 2176, 128, 128, "one"),     # a part of one row, sums of 17
                                                   (129, 1, 2, 1152, 256, 128, "one")])
def test_products_of_few_workgroups(dev, M, k, E, H, I, block_m, how):
    test_gate_up(dev, M, k, E, H, I, block_m, how)
    test_dx_plain(dev, M, k, E, H, I, block_m, how)
    test_dx_through_silu(dev, M, k, E, H, I, block_m, how)


#  256 x 256 tiles, few workgroups' worth of them and more, with rows for several stages
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,k,E,H,I,block_m,how", [(2100, 2, 20, 640, 384, 64, "spread"), (1100, 2, 2, 2432, 1152, 128, "dropped"),
                                                   (700, 1, 9, 1152, 1152, 128, "spread"), (1500, 3, 41, 512, 256, 64, "one"),
                                                   (1401, 3, 21, 640, 384, 128, "dropped"), (1400, 3, 21, 384, 640, 1, "one")])
def test_dw_of_more_rows(dev, M, k, E, H, I, block_m, how, dtype):
    test_dw(dev, M, k, E, H, I, block_m, how, dtype)


def test_silu_gradient_past_four_gib(dev):
    """z and its gradients of 70000 x 32768 (4.6 GB each): rows and columns from their far ends."""
    import moe_layer_topk_amd as moe
    M, H, I = 70000, 128, 16384
    al = moe.moe_align(torch.zeros(M, 1, dtype=torch.int32, device=dev), 1, 128)
    g = torch.Generator(device=dev).manual_seed(10)
    z = torch.empty(M, 2 * I, dtype=BF, device=dev)
    for i in range(0, M, 10000):
        z[i:i + 10000] = torch.randn(10000, 2 * I, generator=g, device=dev).to(BF)
    assert z.numel() * 2 > 2 ** 32
    w = (torch.randn(1, H, I, generator=g, device=dev) * 0.05).to(BF)
    dy = torch.randn(M, H, generator=g, device=dev).to(BF)
    da, act = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy, w, al, M, 1, z=z)
    for r in (slice(0, 3), slice(33333, 33336), slice(M - 3, M)):
        a, b = dy[r].cpu().double(), w[0].cpu().double()
        d, e_d = a @ b, 2 * H * U * (a.abs() @ b.abs())
        want, wact, slope, mag = silu_grad(d, z[r].cpu().double())
        close(da[r], want, HALF[BF] * want.abs() + torch.cat([e_d, e_d], 1) * slope * 1.01 + 16 * U * mag + 1e-38, "dz")
        close(act[r], wact, (HALF[BF] + 16 * U) * wact.abs() + 1e-38, "act")


def test_large_dw_tiles_past_four_gib(dev):
    """dc of 70000 x 32768 (4.6 GB) against 384 columns: 256 tiles of 256 x 256, whose rows
    and columns lie past 32 bits (test_operands_past_four_gib has few enough for the
    smaller ones)."""
    import moe_layer_topk_amd as moe
    M, N, K = 70000, 32768, 384
    al = moe.moe_align(torch.zeros(M, 1, dtype=torch.int32, device=dev), 1, 128)
    g = torch.Generator(device=dev).manual_seed(11)
    dc = torch.empty(M, N, dtype=BF, device=dev)
    for i in range(0, M, 10000):
        dc[i:i + 10000] = torch.randn(10000, N, generator=g, device=dev).to(BF)
    a = torch.randn(M, K, generator=g, device=dev).to(BF)
    for kind in (moe.MOE_GEMM_DOWN, moe.MOE_GEMM_GATE_UP):
        dw = moe.moe_grouped_gemm_dw(kind, dc, a, al, M, 1, dtype=F32)
        for c in (slice(0, 3), slice(16383, 16386), slice(N - 3, N)):
            d, v = dc[:, c].double(), a.double()
            want = d.t() @ v
            close(dw[0, c], want.cpu(), (HALF[F32] * want.abs() + 2 * M * U * (d.abs().t() @ v.abs())).cpu(), "dw")
