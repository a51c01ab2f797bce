"""Refusals of the calls around the experts and of the gradients (host checks only; no
GPU needed)."""
import ctypes
import os

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: validation fails first
ELSE = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10004)
NULL = None


@pytest.fixture(scope="module")
def L():
    from moe_layer_topk_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from moe_layer_topk_amd import build
        build.build()
    return _lib.lib()


@pytest.fixture(scope="module")
def bal():
    from moe_layer_topk_amd._lib import AlignBufs
    return ctypes.byref(AlignBufs(*(0x10000,) * 6))


def test_permute(L, bal):
    from moe_layer_topk_amd._lib import AlignBufs

    def f(dt=1, x=FAKE, w=NULL, ids=FAKE, al=bal, M=4, k=2, E=8, bm=16, H=64, rows=FAKE, at=FAKE):
        return L.moe_permute(dt, x, w, ids, al, M, k, E, bm, H, rows, at, NULL)

    assert f(M=0, x=NULL, ids=NULL, al=None, rows=NULL, at=NULL) == 0
    assert f(dt=2) == 3
    assert f(H=60) == 2
    assert f(H=0) == 2
    assert f(M=-1) == 2
    assert f(k=9) == 2
    assert f(k=17, E=64) == 3
    assert f(E=257) == 3
    assert f(bm=24) == 3
    assert f(M=(1 << 23) + 1, k=1) == 3
    assert f(M=1 << 24, k=2) == 3
    for bad in (dict(x=NULL), dict(ids=NULL), dict(al=None), dict(rows=NULL), dict(at=NULL)):
        assert f(**bad) == 1
    for bad in (dict(x=ODD), dict(w=ODD), dict(ids=ODD), dict(rows=ODD), dict(at=ODD)):
        assert f(**bad) == 5
    assert f(al=ctypes.byref(AlignBufs(0x10000, 0, 0x10000, 0x10000, 0x10000, 0x10000))) == 1
    assert f(al=ctypes.byref(AlignBufs(0x10004, 0x10000, 0x10000, 0x10000, 0x10000, 0x10000))) == 5


def test_unpermute(L):
    def f(dt=1, rows=FAKE, n=8, at=FAKE, w=NULL, M=4, k=2, H=64, odt=1, out=FAKE):
        return L.moe_unpermute(dt, rows, n, at, w, M, k, H, odt, out, NULL)

    assert f(M=0, rows=NULL, out=NULL, n=0) == 0
    assert f(dt=3) == 3
    assert f(odt=2) == 3
    assert f(H=4) == 2
    assert f(k=0) == 2
    assert f(k=17) == 3
    assert f(n=-1) == 2
    assert f(n=(1 << 28) + 1) == 3
    assert f(at=NULL, n=9) == 2     # pair order has M topk rows
    assert f(rows=NULL) == 1
    assert f(out=NULL) == 1
    assert f(at=ODD) == 5
    assert f(w=ODD) == 5


def test_row_gradients(L, bal):
    def u(dt=1, d=FAKE, rows=FAKE, n=128, at=FAKE, w=FAKE, al=None, M=4, k=2, E=8, bm=16, H=64, o=FAKE, dw=FAKE):
        return L.moe_unpermute_backward(dt, d, rows, n, at, w, al, M, k, E, bm, H, o, dw, NULL)

    assert u(M=0, d=NULL, rows=NULL, o=NULL, dw=NULL, n=0) == 0
    assert u(dt=4) == 3
    assert u(H=9) == 2
    assert u(w=NULL) == 3                      # a gradient of weights that are not there
    assert u(rows=NULL) == 1                   # ... or without rows
    assert u(dw=NULL) == 1
    assert u(d=NULL) == 1
    assert u(o=NULL) == 1
    assert u(at=NULL) == 2                     # 128 rows are not 8 pairs
    assert u(al=bal, n=127) == 2               # the alignment's rows are 128
    assert u(al=bal, at=NULL, n=8) == 2        # pair order has no padding
    assert u(al=bal, bm=5) == 3
    assert u(al=bal, E=300) == 3
    assert u(o=ODD) == 5
    assert u(dw=ODD) == 5

    def p(dt=0, d=FAKE, n=8, at=FAKE, x=FAKE, w=FAKE, M=4, k=2, H=64, o=FAKE, dw=FAKE):
        return L.moe_permute_backward(dt, d, n, at, x, w, M, k, H, o, dw, NULL)

    assert p(M=0, d=NULL, x=NULL, o=NULL, dw=NULL, n=0) == 0
    assert p(dt=2) == 3
    assert p(w=NULL) == 3
    assert p(x=NULL) == 1
    assert p(dw=NULL) == 1
    assert p(d=NULL) == 1
    assert p(o=NULL) == 1
    assert p(at=NULL, n=7) == 2
    assert p(x=ODD) == 5


def spec(post=0x10000, gate=0x10000, pre=0x10000, wdt=1, per_token=0, scale=1.0, eps=1e-6):
    from moe_layer_topk_amd._lib import NormSpec
    return ctypes.byref(NormSpec(post, gate, pre, wdt, per_token, scale, eps))


def test_residual_norm(L):
    def f(s=None, dt=1, h=FAKE, y=FAKE, M=4, H=64, o=FAKE, x=ELSE):
        return L.moe_residual_norm(dt, h, y, spec() if s is None else s, M, H, o, x, NULL)

    assert f(M=0, h=NULL, o=NULL, x=NULL) == 0
    assert L.moe_residual_norm(1, FAKE, FAKE, None, 4, 64, FAKE, ELSE, NULL) == 1
    assert f(dt=2) == 3
    assert f(spec(wdt=2)) == 3
    assert f(H=68) == 2
    assert f(H=16392) == 3
    assert f(M=-1) == 2
    assert f(M=1 << 22) == 3
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert f(spec(**bad)) == 2
    assert f(y=NULL) == 3                                    # a gate of no block
    assert f(spec(None, None), y=NULL) == 3                  # h_out would be h
    assert f(spec(None, None, None), y=NULL, o=NULL, x=NULL) == 1  # nothing to write
    assert f(spec(pre=None)) == 1                            # x without its weight
    assert f(x=NULL) == 1
    assert f(o=NULL) == 1
    assert f(h=NULL) == 1
    assert f(x=FAKE) == 3                                    # h_out and x in one place
    assert f(spec(post=0x10004)) == 5
    assert f(h=ODD) == 5
    assert f(x=ODD) == 5


def test_residual_norm_backward(L):
    n = L.moe_residual_norm_workspace_size(4, 64)
    assert n > 0 and L.moe_residual_norm_workspace_size(0, 64) == 0

    def f(s=None, dt=1, h=FAKE, d=FAKE, dx=FAKE, y=FAKE, M=4, H=64, dh=FAKE, dy=ELSE, a=FAKE, b=FAKE, c=FAKE, ws=FAKE, size=n):
        return L.moe_residual_norm_backward(dt, h, d, dx, y, spec() if s is None else s, M, H, dh, dy, a, b, c, ws, size, NULL)

    assert f(dt=3) == 3
    assert f(spec(post=None)) == 3                           # a gradient of a weight that is not there
    assert f(spec(gate=None)) == 3
    assert f(spec(pre=None), dx=NULL) == 3
    assert f(spec(pre=None), c=NULL) == 1                    # dx without its weight
    assert f(dx=NULL) == 1
    assert f(h=NULL) == 1
    assert f(dh=NULL) == 1
    assert f(dy=NULL) == 1
    assert f(spec(None, None), y=NULL, a=NULL, b=NULL) == 1  # dy of no block
    assert f(ws=NULL) == 1
    assert f(size=n - 1) == 4
    assert f(ws=ctypes.c_void_p(0x10010)) == 5
    assert f(a=ODD) == 5
    assert f(dh=ELSE) == 3
    assert f(d=ODD) == 5
    assert f(M=0, a=NULL, b=NULL, c=NULL, h=NULL, dh=NULL, ws=NULL) == 0


def test_gate_up(L, bal):
    def g(dt=1, a=FAKE, sa=NULL, w=FAKE, M=4, k=2, E=8, N=512, K=256, bm=64, c=FAKE, al=bal):
        return L.moe_grouped_gemm(4, dt, a, sa, w, NULL, al, M, k, E, N, K, bm, c, NULL, NULL)

    assert g(M=0, a=NULL, w=NULL, c=NULL, al=None) == 0
    for dt in (0, 2, 3, 4):
        assert g(dt=dt) == 3
    assert g(N=384) == 2
    assert g(K=200) == 2
    assert g(bm=16) == 3
    assert g(bm=256) == 3
    assert g(sa=FAKE) == 3
    assert g(N=1 << 20, K=4096) == 3
    assert g(a=NULL) == 1
    assert g(c=ODD) == 5


def test_dx(L, bal):
    def f(kind=1, dt=1, dc=FAKE, w=FAKE, z=NULL, al=bal, M=4, k=2, E=8, N=512, K=256, bm=64, da=FAKE, act=NULL):
        return L.moe_grouped_gemm_dx(kind, dt, dc, w, z, al, M, k, E, N, K, bm, da, act, NULL)

    assert f(M=0, dc=NULL, w=NULL, al=None, da=NULL) == 0
    for kind in (0, 2, 3, 5):
        assert f(kind=kind) == 3
    for dt in (0, 2, 3, 4):
        assert f(dt=dt) == 3
    assert f(N=64) == 2
    assert f(K=320) == 2
    assert f(kind=4, N=384) == 2
    assert f(bm=32) == 3
    assert f(bm=0) == 3
    assert f(N=1 << 16, K=1 << 15) == 3        # one expert's weights reach 4 GiB
    assert f(kind=4, z=FAKE) == 3              # SiLU-and-mul lies behind the down product
    assert f(act=FAKE) == 3                    # act comes from z
    assert f(dc=NULL) == 1
    assert f(w=NULL) == 1
    assert f(da=NULL) == 1
    assert f(al=None) == 1
    assert f(z=ODD) == 5
    assert f(da=ODD) == 5


def test_dx_up_to_its_largest_expert(L, bal):
    """4 GiB less 64 KiB of weights are taken (the next argument is looked at), one more
    step of either size is not."""
    def f(N, K):
        return L.moe_grouped_gemm_dx(1, 1, NULL, FAKE, NULL, bal, 4, 2, 8, N, K, 64, FAKE, NULL, NULL)

    assert 2 * 128 * 65535 * 256 == 2 ** 32 - 2 ** 16
    assert f(128 * 65535, 256) == 1
    assert f(256, 128 * 65535) == 1
    assert f(128 * 131071, 128) == 3
    assert f(128, 128 * 131071) == 3
    assert f(128 * 65536, 256) == 3


def test_dw(L, bal):
    def f(kind=1, dt=1, dc=FAKE, a=FAKE, al=bal, M=4, k=2, E=8, N=512, K=256, bm=64, odt=1, dw=FAKE):
        return L.moe_grouped_gemm_dw(kind, dt, dc, a, al, M, k, E, N, K, bm, odt, dw, NULL)

    for kind in (0, 2, 3, 5):
        assert f(kind=kind) == 3
    assert f(dt=0) == 3
    assert f(odt=2) == 3
    assert f(N=100) == 2
    assert f(kind=4, N=384) == 2
    assert f(bm=48) == 3
    assert f(dc=NULL) == 1
    assert f(a=NULL) == 1
    assert f(dw=NULL) == 1
    assert f(dw=NULL, M=0) == 1                # an empty batch still clears dw
    assert f(al=None) == 1
    assert f(a=ODD) == 5
    assert f(dw=ODD) == 5


def test_binding_refusals():
    import moe_layer_topk_amd as moe
    t, b = torch.zeros(4, 64), torch.zeros(4, 128, dtype=torch.bfloat16)
    at = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: moe.moe_permute(t, at, {}), lambda: moe.moe_unpermute(t, at),
                 lambda: moe.moe_unpermute_backward(t, t, torch.zeros(4, 1)), lambda: moe.moe_permute_backward(t, at),
                 lambda: moe.moe_residual_norm(t, t), lambda: moe.moe_residual_norm_backward(t, t),
                 lambda: moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, b, torch.zeros(1, 128, 128), {}, 4, 1),
                 lambda: moe.moe_grouped_gemm_dw(moe.MOE_GEMM_DOWN, b, b, {"expert_counts": at}, 4, 1),
                 lambda: moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, b, torch.zeros(1, 256, 128, dtype=torch.bfloat16), {}, 4, 1)):
        with pytest.raises(ValueError, match="GPU only"):
            call()


def test_gate_up_has_no_scales():
    import moe_layer_topk_amd as moe
    b, w, s = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(1, 256, 128, dtype=torch.bfloat16), torch.ones(1)
    for more in (dict(a_scale=s), dict(w_scale=s), dict(c_amax=s)):
        with pytest.raises(ValueError, match="scale"):
            moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, b, w, {}, 4, 1, **more)
