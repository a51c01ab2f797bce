"""The norms around a block with its gate and residual scale, and their gradients,
against float64.

Bounds: a float32 sum over a row is formed as a tree of at most 64 additions in a
line (16 in a thread, 6 across a wavefront, 16 across wavefronts, and the spare),
so a mean square is off by 64 U of itself and a normed value by 40 U more or less;
64 U covers a normed value, and every float32 product or sum after it adds U of the
magnitudes that meet in it.  An output adds its own rounding."""
import pytest
import torch

import train_ref as ref
from train_ref import HALF, U, close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


#        M    H     dtype wdtype block post  gate      pre
CASES = [(1, 8, F32, F32, True, True, "channel", True),
         (1, 4096, BF, BF, True, True, "token", True),
         (5, 64, BF, F32, True, False, "none", True),
         (3, 520, F32, BF, True, True, "token", False),
         (130, 2048, BF, BF, True, True, "channel", True),
         (67, 2056, BF, BF, False, False, "none", True),
         (40, 4104, F32, F32, True, False, "channel", True),
         (9, 8192, BF, F32, True, True, "none", True),
         (4, 16384, F32, F32, True, True, "token", True),
         (4, 16376, BF, BF, True, True, "channel", False),
         (1300, 264, BF, BF, True, True, "channel", True),
         (700, 512, F32, F32, True, False, "token", True),
         (300, 1024, F32, F32, True, True, "channel", True),
         (521, 512, BF, F32, True, False, "channel", True),
         (257, 4096, F32, BF, True, True, "none", True),
         (600, 4096, BF, BF, True, True, "channel", True),
         (3, 12288, BF, F32, True, True, "token", True)]


def make(M, H, dtype, wdtype, block, post, gate, pre, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, size=1.0, to=dtype):
        return (torch.randn(*shape, generator=g) * size).to(to)

    return dict(h=r(M, H, size=2.0), y=r(M, H) * torch.exp(r(M, 1, to=F32)).to(dtype) if block else None,
                post=1 + r(H, size=0.2, to=F32) if post else None,
                gate={"none": None, "channel": r(H, to=F32), "token": r(M, 1, to=F32)}[gate],
                pre=1 + r(H, size=0.2, to=F32) if pre else None, scale=-0.7 if block else 1.0,
                dh_out=r(M, H), dx=r(M, H) if pre else None, wdtype=wdtype)


def weights(c, dev):
    return dict(post_weight=None if c["post"] is None else c["post"].to(c["wdtype"]).to(dev),
                gate=None if c["gate"] is None else c["gate"].to(c["wdtype"]).to(dev),
                pre_weight=None if c["pre"] is None else c["pre"].to(c["wdtype"]).to(dev), scale=c["scale"], eps=EPS)


def on(dev, t):
    return None if t is None else t.to(dev)


def f64(c):
    d = {k: None if c[k] is None else c[k].double() for k in ("h", "y", "dh_out", "dx")}
    d.update({k: None if c[k] is None else c[k].to(c["wdtype"]).double() for k in ("post", "gate", "pre")})
    d["scale"] = float(torch.tensor(c["scale"], dtype=F32))
    return d


def forward_bounds(d, out, x, dtype):
    """Bounds of h_out and x from the magnitudes that meet in them."""
    step = (out - d["h"]).abs()
    e_out = (64 + 6) * U * step + U * (out.abs() + d["h"].abs())
    b_out = HALF[dtype] * out.abs() + e_out
    if x is None:
        return b_out, None
    r = 1 / torch.sqrt((out * out).mean(1, keepdim=True) + EPS)
    # the mean square moves by at most twice the row's relative error, the root by once
    row = e_out.norm(dim=1, keepdim=True) / out.norm(dim=1, keepdim=True).clamp(min=1e-30)
    e_x = (d["pre"].abs() * r) * e_out + x.abs() * (row + (64 + 4) * U)
    return b_out, (HALF[dtype] * x.abs() + 1.01 * e_x)


@pytest.mark.parametrize("M,H,dtype,wdtype,block,post,gate,pre", CASES)
def test_forward(dev, M, H, dtype, wdtype, block, post, gate, pre):
    import moe_layer_topk_amd as moe
    c = make(M, H, dtype, wdtype, block, post, gate, pre, 1)
    if M > 2:  # rows of zeros: the norm of nothing is 0
        c["h"][1] = 0
        if block:
            c["y"][1] = 0
    h = c["h"].to(dev)
    h_out, x = moe.moe_residual_norm(h, on(dev, c["y"]), **weights(c, dev))
    d = f64(c)
    want, wx = ref.residual_norm(d["h"], d["y"], d["post"], d["gate"], d["scale"], d["pre"], EPS)
    b_out, b_x = forward_bounds(d, want, wx, dtype)
    if block:
        close(h_out, want, b_out, "h_out")
    else:
        assert h_out is h
    if pre:
        close(x, wx, b_x, "x")
    else:
        assert x is None
    # in place: h_out over h and x over y, or the other way round
    if block:
        for swap in (False, True):
            h2, y2 = c["h"].to(dev), c["y"].to(dev)
            a, b = (y2, h2) if swap else (h2, y2)
            moe.moe_residual_norm(h2, y2, **weights(c, dev), h_out=a, x=b if pre else None)
            assert torch.equal(a, h_out) and (not pre or torch.equal(b, x))


@pytest.mark.parametrize("M,H,dtype,wdtype,block,post,gate,pre", CASES)
def test_backward(dev, M, H, dtype, wdtype, block, post, gate, pre):
    import moe_layer_topk_amd as moe
    c = make(M, H, dtype, wdtype, block, post, gate, pre, 2)
    kw = weights(c, dev)
    args = [on(dev, c[k]) for k in ("h", "dh_out", "dx", "y")]  # h stands for h_out
    dh, dy, dpost, dgate, dpre = moe.moe_residual_norm_backward(*args, **kw)
    d = f64(c)
    # dh' = dh_out + r2 (q - n mean(q n)), q = dx w_pre, n = h' r2
    want, mag = d["dh_out"], d["dh_out"].abs()
    if pre:
        r2 = 1 / torch.sqrt((d["h"] ** 2).mean(1, keepdim=True) + EPS)
        n, q = d["h"] * r2, d["dx"] * d["pre"]
        want = want + r2 * (q - n * (q * n).mean(1, keepdim=True))
        mag = mag + r2 * (q.abs() + n.abs() * (q * n).abs().mean(1, keepdim=True))
        close(dpre, (d["dx"] * n).sum(0), (M + 64 + 8) * U * (d["dx"] * n).abs().sum(0), "dpre_weight")
    else:
        assert dpre is None
    close(dh, want, HALF[dtype] * want.abs() + 160 * U * mag, "dh")
    if not block:
        assert dy is None and dpost is None and dgate is None
        return
    s = d["scale"]
    r1 = 1 / torch.sqrt((d["y"] ** 2).mean(1, keepdim=True) + EPS) if post else torch.ones(M, 1, dtype=torch.float64)
    n = d["y"] * r1
    u = n * d["post"] if post else n
    g = 1.0 if d["gate"] is None else d["gate"]
    du, du_m = s * want * g, (s * mag * g).abs()  # (mag: what the error of dh' is measured by)
    if gate == "channel":
        close(dgate, (s * want * u).sum(0), (M + 64 + 250) * U * (s * mag * u).abs().sum(0), "dgate")
    elif gate == "token":
        assert dgate.shape == (M, 1)
        close(dgate, (s * want * u).sum(1, keepdim=True), (64 + 250) * U * (s * mag * u).abs().sum(1, keepdim=True), "dgate")
    else:
        assert dgate is None
    if post:
        close(dpost, (du * n).sum(0), (M + 64 + 250) * U * (du_m * n).abs().sum(0), "dpost_weight")
        q, q_m = du * d["post"], (du_m * d["post"]).abs()
        wy = r1 * (q - n * (q * n).mean(1, keepdim=True))
        y_m = r1 * (q_m + n.abs() * (q_m * n.abs()).mean(1, keepdim=True))
    else:
        assert dpost is None
        wy, y_m = du, du_m
    close(dy, wy, HALF[dtype] * wy.abs() + 400 * U * y_m, "dy")
    # in place, and the same bits again
    dh2, dy2 = c["dh_out"].to(dev), c["y"].to(dev)
    again = moe.moe_residual_norm_backward(args[0], dh2, args[2], dy2, **kw, dh=dh2, dy=dy2)
    for a, b in zip((dh, dy, dpost, dgate, dpre), again):
        assert a is None or torch.equal(a, b)


def test_no_gradient_of_the_stream(dev):
    """dh_out None is a gradient of zero."""
    import moe_layer_topk_amd as moe
    c = make(30, 1024, BF, BF, True, True, "channel", True, 3)
    kw = weights(c, dev)
    a = moe.moe_residual_norm_backward(c["h"].to(dev), None, c["dx"].to(dev), c["y"].to(dev), **kw)
    b = moe.moe_residual_norm_backward(c["h"].to(dev), torch.zeros(30, 1024, dtype=BF, device=dev), c["dx"].to(dev),
                                       c["y"].to(dev), **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("post,gate", [(True, "channel"), (False, "token"), (True, "token")])
def test_gradients_against_differences(dev, post, gate):
    """Central differences of the float64 form along random directions against the
    kernels' gradients in float32: a step of 1e-4 leaves 1e-8 of curvature, the
    kernels 400 U of the magnitudes (2.4e-5)."""
    import moe_layer_topk_amd as moe
    c = make(6, 96, F32, F32, True, post, gate, True, 4)
    d = f64(c)
    names = [k for k in ("h", "y", "post", "gate", "pre") if d[k] is not None]
    with torch.no_grad():
        out, _ = ref.residual_norm(d["h"], d["y"], d["post"], d["gate"], d["scale"], d["pre"], EPS)
    got = moe.moe_residual_norm_backward(out.float().to(dev), c["dh_out"].to(dev), c["dx"].to(dev), c["y"].to(dev),
                                         **weights(c, dev))
    grad = dict(h=got[0], y=got[1], post=got[2], gate=got[3], pre=got[4])

    def loss(**over):
        a = {**d, **over}
        o, x = ref.residual_norm(a["h"], a["y"], a["post"], a["gate"], a["scale"], a["pre"], EPS)
        return float((o * d["dh_out"]).sum() + (x * d["dx"]).sum())

    g = torch.Generator().manual_seed(5)
    for k in names:
        v = torch.randn(d[k].shape, generator=g, dtype=torch.float64)
        diff = (loss(**{k: d[k] + 1e-4 * v}) - loss(**{k: d[k] - 1e-4 * v})) / 2e-4
        along = grad[k].double().cpu() * v
        assert abs(diff - float(along.sum())) <= 1e-4 * float(along.abs().sum()), k


def test_infinities_and_nans_stay_in_their_rows(dev):
    import moe_layer_topk_amd as moe
    c = make(6, 256, BF, BF, True, True, "none", True, 6)
    clean = moe.moe_residual_norm(c["h"].to(dev), c["y"].to(dev), **weights(c, dev))
    c["h"][2, 5], c["y"][4, 7] = float("inf"), float("nan")
    out, x = moe.moe_residual_norm(c["h"].to(dev), c["y"].to(dev), **weights(c, dev))
    for t in (0, 1, 3, 5):
        assert torch.equal(out[t], clean[0][t]) and torch.equal(x[t], clean[1][t])
    assert torch.isinf(out[2, 5]) and torch.isnan(x[2, 5])
    assert torch.isnan(out[4]).all() and torch.isnan(x[4]).all()


def test_empty_batch(dev):
    import moe_layer_topk_amd as moe
    e, w = torch.empty(0, 64, device=dev), torch.ones(64, device=dev)
    h, x = moe.moe_residual_norm(e, e.clone(), post_weight=w, gate=w, pre_weight=w)
    assert h.shape == x.shape == (0, 64)
    dh, dy, dpost, dgate, dpre = moe.moe_residual_norm_backward(e, e.clone(), e.clone(), e.clone(), post_weight=w, gate=w,
                                                                pre_weight=w)
    assert dh.shape == dy.shape == (0, 64)
    for t in (dpost, dgate, dpre):  # sums over no rows
        assert torch.equal(t, torch.zeros(64, device=dev))
    g = torch.empty(0, 1, device=dev)
    assert moe.moe_residual_norm_backward(e, e.clone(), None, e.clone(), gate=g)[3].shape == (0, 1)


def test_rows_past_four_gib(dev):
    import moe_layer_topk_amd as moe
    M, H = 300000, 8192
    h = torch.zeros(M, H, dtype=BF, device=dev)
    g = torch.Generator().manual_seed(7)
    for t in (0, 149999, M - 1):
        h[t] = torch.randn(H, generator=g).to(dev)
    w = torch.ones(H, device=dev, dtype=BF)
    assert h.numel() * 2 > 2 ** 32
    _, x = moe.moe_residual_norm(h, pre_weight=w, x=h.clone())
    for t in (0, 149999, M - 1):
        v = h[t].double().cpu()
        want = v / torch.sqrt((v * v).mean() + EPS)
        close(x[t], want, want.abs() * (HALF[BF] + 70 * U), f"row {t}")
    assert not x[1].any() and not x[M - 2].any()


def test_graphs(dev):
    """A captured step replayed with the program's own work between."""
    import moe_layer_topk_amd as moe
    c = make(600, 2048, BF, BF, True, True, "channel", True, 8)
    kw = weights(c, dev)
    h, y, dh_out, dx = (c[k].to(dev) for k in ("h", "y", "dh_out", "dx"))
    bufs = [torch.empty_like(h) for _ in range(4)]
    ws = torch.empty(moe.lib().moe_residual_norm_workspace_size(600, 2048), dtype=torch.uint8, device=dev)

    def step():
        moe.moe_residual_norm(h, y, **kw, h_out=bufs[0], x=bufs[1])
        return moe.moe_residual_norm_backward(bufs[0], dh_out, dx, y, **kw, dh=bufs[2], dy=bufs[3], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    g = torch.Generator().manual_seed(9)
    for _ in range(4):
        y.copy_(torch.randn(600, 2048, generator=g).bfloat16())
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*bufs, *held[2:])]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*bufs, *eager[2:])))


#  What the cases above leave out: every way a row is held (threads, pieces a thread, rows
#  that fill their workgroup or not), each with more rows than workgroups, so that sums go
#  on from row to row, the shared buffers alternate and the next row is on its way.
#  (Long rows add 32 values in a thread, 6 times across a wavefront and 8 wavefronts: 46
#  in a line, under the 64 above.)
#        M    H     dtype wdtype block post  gate      pre
MORE = [(300, 1000, BF, BF, True, True, "channel", True),      # 128 threads
        (520, 1024, BF, F32, True, True, "none", True),
        (1030, 1032, BF, BF, True, True, "token", True),       # 256
        (600, 2040, BF, BF, True, True, "channel", True),
        (520, 2048, BF, F32, True, False, "channel", True),
        (600, 4088, BF, BF, True, True, "token", True),        # 512
        (300, 4104, BF, BF, True, True, "channel", True),      # 1024
        (600, 5120, BF, F32, True, True, "channel", True),
        (520, 6144, BF, BF, True, True, "token", True),
        (515, 7168, BF, BF, False, False, "none", True),
        (600, 8184, BF, BF, True, False, "none", False),
        (600, 8192, BF, BF, True, True, "channel", True),
        (600, 8200, BF, BF, True, True, "token", True),        # long rows
        (530, 12288, BF, F32, True, True, "channel", True),
        (600, 16384, BF, BF, True, True, "channel", True),
        (600, 248, F32, F32, True, True, "channel", True),     # 64
        (300, 256, F32, BF, True, True, "none", True),
        (520, 512, F32, F32, True, True, "channel", True),     # 128
        (600, 1016, F32, F32, True, True, "token", True),      # 256
        (520, 1032, F32, F32, True, True, "channel", True),    # 512
        (600, 2040, F32, BF, True, True, "token", True),
        (1100, 2048, F32, F32, True, True, "channel", True),
        (600, 2056, F32, F32, True, True, "channel", True),    # 1024
        (520, 4088, F32, BF, True, False, "token", True),
        (600, 4096, F32, F32, True, True, "channel", True),
        (600, 4104, F32, F32, True, True, "channel", True),    # long rows
        (520, 8192, F32, BF, True, True, "token", True),
        (520, 8200, F32, F32, True, True, "token", True),
        (600, 16384, F32, F32, True, True, "channel", True)]


@pytest.mark.parametrize("M,H,dtype,wdtype,block,post,gate,pre", MORE)
def test_every_way_a_row_is_held(dev, M, H, dtype, wdtype, block, post, gate, pre):
    test_forward(dev, M, H, dtype, wdtype, block, post, gate, pre)
    test_backward(dev, M, H, dtype, wdtype, block, post, gate, pre)


def test_long_rows_over_every_input(dev):
    """Rows of several pieces a thread over each of their inputs: the same bits as apart."""
    import moe_layer_topk_amd as moe
    for H, dtype in ((12288, BF), (4104, F32), (16384, F32)):
        c = make(560, H, dtype, dtype, True, True, "channel", True, 21)
        kw = weights(c, dev)
        names = ("h", "dh_out", "dx", "y")
        apart = moe.moe_residual_norm_backward(*(c[k].to(dev) for k in names), **kw)
        for over in ((0, 1), (1, 2), (2, 3), (3, 0)):
            args = [c[k].to(dev) for k in names]
            got = moe.moe_residual_norm_backward(*args, **kw, dh=args[over[0]], dy=args[over[1]])
            assert all(torch.equal(a, b) for a, b in zip(apart, got)), (H, over)


def test_gradients_of_rows_past_four_gib(dev):
    """Rows from both ends and the middle of 4.9 GB tensors, zeros elsewhere: the bits of a
    row alone (a row's sums are its own), and column sums that add just those rows."""
    import moe_layer_topk_amd as moe
    M, H, at = 300000, 8192, [0, 149999, 299999]
    c = make(3, H, BF, BF, True, True, "channel", True, 22)
    kw = weights(c, dev)
    big = {}
    for name in ("h", "dh_out", "dx", "y"):
        big[name] = torch.zeros(M, H, dtype=BF, device=dev)
        big[name][at] = c[name].to(dev)
    assert big["h"].numel() * 2 > 2 ** 32
    alone = [moe.moe_residual_norm_backward(*(c[n][i:i + 1].to(dev) for n in ("h", "dh_out", "dx", "y")), **kw)
             for i in range(3)]
    dh, dy, *sums = moe.moe_residual_norm_backward(big["h"], big["dh_out"], big["dx"], big["y"], **kw, dh=big["dh_out"],
                                                   dy=big["dx"])
    for i, t in enumerate(at):
        assert torch.equal(dh[t], alone[i][0][0]) and torch.equal(dy[t], alone[i][1][0]), t
    for t in (1, 149998, 150000, M - 2):
        assert not dh[t].any() and not dy[t].any()
    for j, got in enumerate(sums):
        parts = torch.stack([a[2 + j].double().cpu() for a in alone])
        # (two float32 sums in any order; dpost and dgate are S times a weight on either side: 2 more)
        close(got, parts.sum(0), 5 * U * parts.abs().sum(0), f"sum {j}")
    # a gate a token: the form with conditions
    kw["gate"] = torch.ones(M, 1, dtype=BF, device=dev)
    g1 = torch.ones(1, 1, dtype=BF, device=dev)
    alone = [moe.moe_residual_norm_backward(*(c[n][i:i + 1].to(dev) for n in ("h", "dh_out", "dx", "y")), **{**kw, "gate": g1})
             for i in range(3)]
    for name in ("dh_out", "dx"):
        big[name].zero_()
        big[name][at] = c[name].to(dev)
    dh, dy, _, dgate, _ = moe.moe_residual_norm_backward(big["h"], big["dh_out"], big["dx"], big["y"], **kw, dh=big["dh_out"],
                                                         dy=big["dx"])
    for i, t in enumerate(at):
        assert torch.equal(dh[t], alone[i][0][0]) and torch.equal(dy[t], alone[i][1][0]), t
        assert torch.equal(dgate[t], alone[i][3][0])
    assert int((dgate != 0).sum()) == 3
