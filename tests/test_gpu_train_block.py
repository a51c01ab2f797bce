"""One residual block of a fine-grained layer forward and backward on the framework's
calls, as a training step runs them, against float64 with the same roundings."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


def make(M, E, k, H, I, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape, size=1.0, to=BF):
        return (torch.randn(*shape, generator=g) * size).to(to)

    return dict(h=r(M, H, size=2.0), w_in=(1 + r(H, size=0.1, to=torch.float32)).to(BF),
                w_post=(1 + r(H, size=0.1, to=torch.float32)).to(BF), gate=r(H, size=0.5),
                wr=r(E, H, size=0.05, to=torch.float32), w1=r(E, 2 * I, H, size=0.05), w2=r(E, H, I, size=0.05),
                dout=r(M, H))


def block(moe, p, M, E, k, H, I, scale, sorted_rows):
    """Forward and backward; sorted_rows: through rows in expert order."""
    _, x = moe.moe_residual_norm(p["h"], pre_weight=p["w_in"], eps=EPS)
    logits = moe.moe_router_logits(x, p["wr"])
    ids, wts = moe.moe_route(logits, k)
    al = moe.moe_align(ids, E, 64)
    z, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, p["w1"], al, M, k)
    act, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU, x, p["w1"], al, M, k)
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN, act, p["w2"], al, M, k)
    if sorted_rows:  # the same rows by way of expert order (as another device would hold them)
        one = ids.view(-1, 1)
        al1 = moe.moe_align(one, E, 16)
        rows, at = moe.moe_permute(y, one, al1)
        at = at.view(M, k)
        out = moe.moe_unpermute(rows, at, wts)
    else:
        out = moe.moe_combine(y, wts, k)
    h_out, _ = moe.moe_residual_norm(p["h"], out, post_weight=p["w_post"], gate=p["gate"], scale=scale, eps=EPS)
    # ---- backward
    dh, dout, dpost, dgate, _ = moe.moe_residual_norm_backward(h_out, p["dout"], None, out, post_weight=p["w_post"],
                                                               gate=p["gate"], scale=scale, eps=EPS)
    if sorted_rows:
        drows, dw = moe.moe_unpermute_backward(dout, rows, wts, at, drows=torch.zeros_like(rows))
        dy, _ = moe.moe_permute_backward(drows, at.view(-1, 1))
    else:
        dy, dw = moe.moe_unpermute_backward(dout, y, wts)
    dz, act_b = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy, p["w2"], al, M, k, z=z)
    dw2 = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_DOWN, dy, act_b, al, M, k)
    dxp, _ = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_GATE_UP, dz, p["w1"], al, M, k)
    dw1 = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_GATE_UP, dz, x, al, M, k)
    dx, _ = moe.moe_permute_backward(dxp, topk=k)
    dh_in, _, _, _, dw_in = moe.moe_residual_norm_backward(p["h"], dh, dx, pre_weight=p["w_in"], eps=EPS)
    return dict(ids=ids, wts=wts, x=x, z=z, act=act_b, y=y, out=out, h_out=h_out, dh=dh, dout=dout, dpost=dpost,
                dgate=dgate, dy=dy, dw=dw, dz=dz, dw1=dw1, dw2=dw2, dxp=dxp, dx=dx, dh_in=dh_in, dw_in=dw_in)


def reference(p, got, M, E, k, H, I, scale):
    """Every tensor in float64 from the call's own inputs as the run had them."""
    q = {n: t.double().cpu() for n, t in p.items()}
    v = {n: t.double().cpu() if t.is_floating_point() else t.cpu() for n, t in got.items()}
    flat = v["ids"].reshape(-1)
    want = dict(x=ref.rms_norm(q["h"], EPS) * q["w_in"])
    lists = [(flat == e).nonzero().flatten() for e in range(E)]
    for n, cols in (("z", 2 * I), ("act", I), ("y", H), ("dz", 2 * I), ("dxp", H)):
        want[n] = torch.zeros(M * k, cols, dtype=torch.float64)
    want["dw1"], want["dw2"] = torch.zeros_like(q["w1"]), torch.zeros_like(q["w2"])
    for e, i in enumerate(lists):
        want["z"][i] = v["x"][i // k] @ q["w1"][e].t()
        want["act"][i] = ref.silu_mul(v["z"][i])
        d = v["dy"][i] @ q["w2"][e]
        gt, up = v["z"][i][:, :I], v["z"][i][:, I:]
        s = torch.sigmoid(gt)
        want["dz"][i] = torch.cat([d * up * s * (1 + gt * (1 - s)), d * gt * s], 1)
        want["dxp"][i] = v["dz"][i] @ q["w1"][e]
        want["dw1"][e] = v["dz"][i].t() @ v["x"][i // k]
        want["dw2"][e] = v["dy"][i].t() @ v["act"][i]
        want["y"][i] = v["act"][i] @ q["w2"][e].t()
    yk = v["y"].view(M, k, H)
    want["out"] = (yk * v["wts"][:, :, None]).sum(1)
    want["h_out"], _ = ref.residual_norm(q["h"], v["out"], q["w_post"], q["gate"], scale, None, EPS)
    out = v["out"].clone().requires_grad_()
    post, gate = q["w_post"].clone().requires_grad_(), q["gate"].clone().requires_grad_()
    step, _ = ref.residual_norm(torch.zeros_like(out), out, post, gate, scale, None, EPS)
    want["dout"], want["dpost"], want["dgate"] = torch.autograd.grad(step, (out, post, gate), q["dout"])
    want["dh"] = q["dout"]
    want["dy"] = (v["dout"][:, None, :] * v["wts"][:, :, None]).reshape(M * k, H)
    want["dw"] = (yk * v["dout"][:, None, :]).sum(2)
    want["dx"] = v["dxp"].view(M, k, H).sum(1)
    h, w_in = q["h"].clone().requires_grad_(), q["w_in"].clone().requires_grad_()
    more, want["dw_in"] = torch.autograd.grad(ref.rms_norm(h, EPS) * w_in, (h, w_in), v["dx"])
    want["dh_in"] = v["dh"] + more
    return want, v


@pytest.mark.parametrize("sorted_rows", [False, True])
@pytest.mark.parametrize("M,E,k,H,I", [(1, 8, 2, 256, 128), (75, 16, 4, 384, 256), (260, 4, 2, 512, 384)])
def test_block(dev, M, E, k, H, I, sorted_rows):
    """Each result from the inputs that the run itself had: off by one rounding of the
    result (2^-8 of its norm for bfloat16 rows; sums in float32 1e-5, which is over 400 U
    times the ratio of a sum's magnitudes to its size here).  y comes from the fused
    kind's act, whose z was not rounded: two roundings of z more, silu's slope at most 1.1."""
    import moe_layer_topk_amd as moe
    p = {n: t.to(dev) for n, t in make(M, E, k, H, I, 1).items()}
    got = block(moe, p, M, E, k, H, I, 0.8, sorted_rows)
    want, v = reference(p, got, M, E, k, H, I, 0.8)
    for n, w in want.items():
        rel = float((v[n] - w).norm() / w.norm())
        f32 = n in ("dpost", "dgate", "dw", "dw_in")
        bound = 1e-5 if f32 else 2.0 ** -8 * (4.5 if n == "y" else 1.0)
        assert rel <= bound, f"{n}: {rel} of {bound}"


def test_block_in_a_graph(dev):
    """The whole step captured: replays on new inputs give the eager step's bits."""
    import moe_layer_topk_amd as moe
    M, E, k, H, I = 130, 8, 2, 256, 256
    p = {n: t.to(dev) for n, t in make(M, E, k, H, I, 2).items()}
    block(moe, p, M, E, k, H, I, 0.8, False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block(moe, p, M, E, k, H, I, 0.8, False)
    for i in range(4):
        p["h"].copy_(make(M, E, k, H, I, 3 + i)["h"].to(dev))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in held.items()}
        eager = block(moe, p, M, E, k, H, I, 0.8, False)
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], eager[n]) for n in got)


@pytest.mark.parametrize("M,E,k,H,I", [(2, 3, 2, 128, 128), (75, 16, 4, 384, 256), (260, 4, 2, 512, 384)])
def test_pairs_of_no_expert(dev, M, E, k, H, I):
    """The products' forward and backward in pair order with ids that are no expert (a
    whole token of them among them): with a pair_row of -1 there nothing of the rows that
    the products leave unwritten, here NaN, gets into any result.

    Bounds: a float32 sum of n terms is off by at most n U times the sum of their
    magnitudes, 2 n U for the matrix instructions; results add their own rounding."""
    import moe_layer_topk_amd as moe
    from train_ref import HALF, U, close
    p = {n: t.to(dev) for n, t in make(M, E, k, H, I, 11).items()}
    g = torch.Generator().manual_seed(12)
    P, F32 = M * k, torch.float32
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)
    ids = torch.where(torch.rand(M, k, generator=g) < 0.3, torch.where(torch.rand(M, k, generator=g) < 0.5, -1, E), ids).int()
    ids[1], ids[0, 0] = -1, 0
    ids, wts = ids.to(dev), torch.rand(M, k, generator=g).to(dev)
    held = (ids >= 0) & (ids < E)
    pair_row = torch.where(held, torch.arange(P, dtype=torch.int32, device=dev).view(M, k), -1)
    assert pair_row.dtype == torch.int32
    x, dout = (0.5 * p["h"].float()).to(BF), p["dout"]

    def nan(cols):
        return torch.full((P, cols), float("nan"), dtype=BF, device=dev)

    al = moe.moe_align(ids, E, 64)
    z, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, p["w1"], al, M, k, c=nan(2 * I))
    act, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU, x, p["w1"], al, M, k, c=nan(I))
    y, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN, act, p["w2"], al, M, k, c=nan(H))
    out = moe.moe_unpermute(y, pair_row, wts)
    dy, dwts = moe.moe_unpermute_backward(dout, y, wts, pair_row, drows=nan(H))
    dz, _ = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy, p["w2"], al, M, k, z=z, da=nan(2 * I), act=nan(I))
    dw2 = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_DOWN, dy, act, al, M, k, dtype=F32)
    dxp, _ = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_GATE_UP, dz, p["w1"], al, M, k, da=nan(H))
    dw1 = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_GATE_UP, dz, x, al, M, k, dtype=F32)
    dx, none = moe.moe_permute_backward(dxp, pair_row)
    assert none is None
    lost = ~held.view(-1)
    for t in (z, act, y, dy, dz, dxp):  # unwritten where no expert is, numbers elsewhere
        assert torch.isnan(t[lost]).all() and torch.isfinite(t[~lost]).all()

    at, live = pair_row.cpu(), held.cpu()
    w = wts.cpu().double()
    want, mag = ref.unpermute(y.cpu(), at, wts.cpu())
    close(out, want, HALF[BF] * want.abs() + 2 * (k + 1) * U * mag, "out")
    yk = torch.where(live[:, :, None], y.cpu().double().view(M, k, H), 0.0)
    prod = yk * dout.cpu().double()[:, None, :]
    close(dwts, prod.sum(2), (H + 2) * U * prod.abs().sum(2), "dweights")
    want = (dout.cpu().double()[:, None, :] * w[:, :, None]).view(P, H)[live.view(-1)]
    close(dy[~lost], want, want.abs() * (HALF[BF] * 1.01 + U), "dy")
    want, mag = ref.unpermute(dxp.cpu(), at, None)
    close(dx, want, HALF[BF] * want.abs() + 2 * (k + 1) * U * mag, "dx")
    for t in (out, dx, dwts):
        assert not t[1].any()  # the token with no expert at all
    flat = ids.cpu().view(-1)
    for e in range(E):
        i = (flat == e).nonzero().flatten()
        for got, d, a in ((dw2, dy.cpu()[i], act.cpu()[i]), (dw1, dz.cpu()[i], x.cpu()[i // k])):
            d, a = d.double(), a.double()
            want = d.t() @ a
            close(got[e], want, HALF[F32] * want.abs() + 2 * max(len(i), 1) * U * (d.abs().t() @ a.abs()), f"dw expert {e}")
    dxp[lost] = 0  # the other way: rows of zeros, every pair added
    again, _ = moe.moe_permute_backward(dxp, topk=k)
    assert torch.equal(again, dx)


def test_dw2_is_the_gradient_of_the_y_that_was_made(dev):
    """y = act W2 is linear in W2: over any direction V the differences of <y, dy> are
    exactly <dW2, V> with dW2 = dy^T act of the act that y was made of, to the float32
    sums of the pairs (2 n U of the magnitudes).  The act made again from z is another
    one: off by the roundings of gate and up (silu's slope is at most 1.1), the sums of
    the two products, and both acts' own roundings."""
    import moe_layer_topk_amd as moe
    from train_ref import HALF, U, close
    M, E, k, H, I = 200, 4, 2, 256, 384
    p = {n: t.to(dev) for n, t in make(M, E, k, H, I, 13).items()}
    g = torch.Generator().manual_seed(14)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32).to(dev)
    x, dy = (0.5 * p["h"].float()).to(BF), torch.randn(M * k, H, generator=g).to(BF).to(dev)
    al = moe.moe_align(ids, E, 64)
    z, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, x, p["w1"], al, M, k)
    act, _ = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU, x, p["w1"], al, M, k)
    kept = act.clone()
    _, again = moe.moe_grouped_gemm_dx(moe.MOE_GEMM_DOWN, dy, p["w2"], al, M, k, z=z)
    assert torch.equal(act, kept)  # the forward's act is left alone
    dw2 = moe.moe_grouped_gemm_dw(moe.MOE_GEMM_DOWN, dy, act, al, M, k, dtype=torch.float32)
    flat = ids.view(-1).cpu()
    v = torch.randn(E, H, I, generator=g, dtype=torch.float64)
    for e in range(E):
        i = (flat == e).nonzero().flatten()
        d, a = dy.cpu()[i].double(), act.cpu()[i].double()
        along = ((a @ v[e].t()) * d).sum()  # (y(W2 + s V) - y(W2)) / s against dy
        assert abs(along - (dw2[e].cpu().double() * v[e]).sum()) <= 2 * len(i) * U * ((d.abs().t() @ a.abs()) * v[e].abs()).sum()
    zd, e_z = z.cpu().double(), torch.zeros(M * k, 2 * I, dtype=torch.float64)
    for e in range(E):
        i = (flat == e).nonzero().flatten()
        e_z[i] = 4 * H * U * (x.cpu()[i // k].double().abs() @ p["w1"][e].cpu().double().abs().t())  # (two products' sums)
    size, off = zd.abs(), 1.01 * HALF[BF] * zd.abs() + e_z
    gt, up, d_gt, d_up = size[:, :I], size[:, I:], off[:, :I], off[:, I:]
    a, b = act.cpu().double(), again.cpu().double()
    moved = 1.1 * d_gt * (up + d_up) + (gt + d_gt) * d_up  # (silu itself is at most its argument)
    close(again, a, moved + (1.01 * HALF[BF] + 16 * U) * (a.abs() + b.abs()) + 1e-38, "act")
