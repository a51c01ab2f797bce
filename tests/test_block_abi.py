"""Refusals of the grouped router and of the block-scaled e4m3 calls (host
checks only; no GPU needed)."""
import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10004)
NULL = None
BLOCK = 4


@pytest.fixture(scope="module")
def L():
    from moe_layer_topk_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from moe_layer_topk_amd import build
        build.build()
    return _lib.lib()


def routing(score=1, bias=None, n_groups=8, topk_groups=4, group_top=2, renorm=1, scale=1.0):
    from moe_layer_topk_amd._lib import RoutingArgs
    return ctypes.byref(RoutingArgs(score, bias, n_groups, topk_groups, group_top, renorm, scale))


def test_route_grouped(L):
    f = L.moe_route_grouped
    call = lambda r, M=4, E=256, k=8, dt=0, lg=FAKE, ids=FAKE, w=FAKE: f(dt, lg, r, M, E, k, ids, w, NULL)  # noqa: E731
    assert call(routing(), M=0, lg=NULL, ids=NULL, w=NULL) == 0  # M = 0: no-op
    assert call(None) == 1
    assert call(routing(), lg=NULL) == 1
    assert call(routing(), ids=NULL) == 1
    assert call(routing(), w=NULL) == 1
    assert call(routing(), lg=ODD) == 5
    assert call(routing(bias=0x10002)) == 5
    assert call(routing(), dt=2) == 3
    assert call(routing(), M=-1) == 2
    assert call(routing(), k=0) == 2
    assert call(routing(), k=17) == 3
    assert call(routing(), E=264) == 3
    assert call(routing(score=2)) == 3
    assert call(routing(n_groups=7)) == 2       # not a divisor of E
    assert call(routing(n_groups=0)) == 2
    assert call(routing(topk_groups=0)) == 2
    assert call(routing(topk_groups=9)) == 2
    assert call(routing(group_top=3)) == 2
    assert call(routing(group_top=0)) == 2
    assert call(routing(n_groups=64, topk_groups=1)) == 2                    # 4 experts cannot give 8
    assert call(routing(n_groups=256, topk_groups=8, group_top=1)) == 3      # more groups than the kernel ranks
    assert call(routing(n_groups=256, topk_groups=8, group_top=2)) == 2      # a group of one has no second
    assert call(routing(scale=float("nan"))) == 2
    assert call(routing(scale=float("inf"))) == 2


def test_quant_block(L):
    q = L.moe_quant_block
    assert q(0, NULL, 0, 256, 1, NULL, NULL, NULL) == 0
    assert q(2, FAKE, 4, 256, 1, FAKE, FAKE, NULL) == 3
    assert q(1, FAKE, -1, 256, 1, FAKE, FAKE, NULL) == 2
    assert q(1, FAKE, 4, 200, 1, FAKE, FAKE, NULL) == 2
    assert q(1, FAKE, 4, 0, 1, FAKE, FAKE, NULL) == 2
    assert q(1, FAKE, 4, 256, 64, FAKE, FAKE, NULL) == 3
    assert q(1, NULL, 4, 256, 1, FAKE, FAKE, NULL) == 1
    assert q(1, FAKE, 4, 256, 1, NULL, FAKE, NULL) == 1
    assert q(1, FAKE, 4, 256, 1, FAKE, NULL, NULL) == 1
    assert q(1, FAKE, 4, 256, 1, FAKE, ODD, NULL) == 5


def test_block_gemm(L):
    from moe_layer_topk_amd._lib import AlignBufs
    bal = ctypes.byref(AlignBufs(*(0x10000,) * 6))

    def g(kind, a=FAKE, sa=FAKE, w=FAKE, sw=FAKE, al=bal, M=4, k=2, E=8, N=512, K=256, bm=64, c=FAKE, sc=NULL):
        return L.moe_grouped_gemm(kind, BLOCK, a, sa, w, sw, al, M, k, E, N, K, bm, c, sc, NULL)

    assert g(3, M=0, a=NULL, sa=NULL, w=NULL, sw=NULL, al=None, c=NULL) == 0
    assert g(4) == 3
    assert L.moe_grouped_gemm(3, 1, FAKE, NULL, FAKE, NULL, bal, 4, 2, 8, 512, 256, 64, FAKE, NULL, NULL) == 3  # bf16
    assert L.moe_grouped_gemm(3, 2, FAKE, FAKE, FAKE, FAKE, bal, 4, 2, 8, 512, 256, 64, FAKE, FAKE, NULL) == 3  # e4m3
    assert g(3, N=384, sc=FAKE) == 2             # gate/up: N a multiple of 256
    assert g(2, N=320) == 2
    assert g(2, K=320) == 2
    assert g(2, bm=16) == 3                      # the E4M3 kinds are tiled
    assert g(3, bm=256, sc=FAKE) == 3
    assert g(0, bm=48) == 3
    assert g(2, N=1 << 18, K=1 << 15) == 3       # one expert's codes reach 4 GiB
    assert g(1, sa=FAKE) == 3                    # DOWN over float32 act has no scales
    assert g(2, sc=FAKE) == 3                    # only the e4m3 act has scales to write
    assert g(3) == 1                             # ... and needs the place
    assert g(2, sa=NULL) == 1
    assert g(2, sw=NULL) == 1
    assert g(0, a=NULL) == 1
    assert g(0, al=None) == 1
    assert g(2, sw=ODD) == 5
    assert g(3, sc=ODD) == 5


def test_block_layer(L):
    sz = L.fused_moe_workspace_size(BLOCK, 64, 8, 2, 4096, 14336)
    assert sz >= 128 * 14336 + 128 * 4096 * 2  # codes of act and bfloat16 y at least
    assert L.moe_block_m(BLOCK, 64, 8, 2) in (32, 64, 128)
    assert L.moe_block_m(BLOCK, 0, 8, 2) == 0
    assert L.moe_block_m(9, 64, 8, 2) == 0
    assert L.moe_block_m(1, 64, 8, 9) == 0
    assert L.moe_block_m(1, 4096, 8, 2) == 128

    def f(r, dt=BLOCK, x=FAKE, xs=NULL, s1=FAKE, s2=FAKE, H=4096, ws=FAKE, n=1 << 40, k=2, out=FAKE, M=64, I=14336):
        return L.fused_moe_grouped(dt, x, xs, FAKE, r, FAKE, s1, FAKE, s2, M, 8, k, H, I, out, NULL, NULL, ws, n, NULL)

    r = routing(n_groups=4, topk_groups=2)
    assert f(r, M=0) == 0
    assert f(None) == 1
    assert f(routing()) == 2                     # 8 experts in 8 groups have no second
    assert f(r, dt=5) == 3
    assert f(r, xs=FAKE) == 3                    # x is bfloat16: no scale
    assert f(r, s1=NULL) == 1
    assert f(r, s2=ODD) == 5
    assert f(r, H=4000) == 2
    assert f(r, k=5) == 2                        # two groups of two hold four experts
    assert f(r, out=NULL) == 1
    assert f(r, ws=NULL) == 1
    assert f(r, ws=ctypes.c_void_p(0x10010)) == 5
    assert f(r, n=sz - 1) == 4
    assert f(r, H=1 << 17, I=1 << 14) == 3       # one expert's gate/up codes reach 4 GiB
    # the cache takes the dtype too
    from moe_layer_topk_amd._lib import ExpertWeights
    out = ctypes.c_void_p()
    plain, scaled = ExpertWeights(FAKE, FAKE, None, None), ExpertWeights(FAKE, FAKE, FAKE, FAKE)
    assert L.moe_cache_create(BLOCK, 8, 256, 384, 4, plain, plain, NULL, ctypes.byref(out)) == 1
    assert L.moe_cache_create(BLOCK, 8, 200, 384, 4, scaled, scaled, NULL, ctypes.byref(out)) == 2
    assert L.fused_moe_noalloc(BLOCK, FAKE, None, FAKE, FAKE, None, FAKE, FAKE, 4, 8, 2, 256, 256, 1, FAKE, None, None,
                               NULL) == 1


def test_binding_refusals():
    import torch

    import moe_layer_topk_amd as moe
    with pytest.raises(ValueError, match="score"):
        moe.Routing(score="tanh")
    with pytest.raises(ValueError, match="CPU"):
        moe.Routing(bias=torch.zeros(8))
    with pytest.raises(ValueError, match="GPU only"):
        moe.moe_route_grouped(torch.zeros(4, 8), 2, moe.Routing())
    with pytest.raises(ValueError, match="GPU only"):
        moe.moe_quant_block(torch.zeros(4, 128))
    with pytest.raises(ValueError, match="GPU only"):
        moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN, torch.zeros(8, 128), torch.zeros(2, 128, 128, dtype=torch.float8_e4m3fn),
                             {}, 4, 2, w_scale=torch.zeros(2, 1, 1))
