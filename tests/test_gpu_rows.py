"""Token rows in expert order and back (moe_permute, moe_unpermute and their
gradients) against float64.

Bounds: a copied row is exact; a weighted one is one float32 product and one
rounding; a sum of n float32 terms is off by at most n U times the sum of their
magnitudes (U half a step of float32), whatever its order, and is rounded once."""
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


#        M   k  E    H    block_m dtype weighted
CASES = [(1, 1, 1, 8, 1, BF, False),
         (1, 8, 128, 2048, 16, BF, False),
         (1, 1, 4, 520, 64, F32, True),
         (3, 2, 8, 8, 128, BF, True),
         (77, 8, 128, 2056, 16, BF, True),
         (300, 2, 8, 4096, 128, BF, True),
         (129, 16, 256, 264, 1, F32, True),
         (64, 4, 40, 1000, 32, F32, False),
         (33, 6, 5 + 1, 20008, 64, BF, True),
         (1500, 3, 7, 72, 256, BF, False)]


def make(M, k, E, H, dtype, weighted, dropped, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32)  # an expert may come twice
    if dropped:
        bad = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64)[torch.randint(0, 4, (M, k), generator=g)]
        ids = torch.where(torch.rand(M, k, generator=g) < 0.2, bad.int(), ids)
    x = torch.randn(M, H, generator=g).to(dtype)
    w = torch.rand(M, k, generator=g) if weighted else None
    return ids, x, w, g


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("M,k,E,H,block_m,dtype,weighted", CASES)
def test_permute(dev, M, k, E, H, block_m, dtype, weighted, dropped):
    import moe_layer_topk_amd as moe
    ids, x, w, _ = make(M, k, E, H, dtype, weighted, dropped, 1)
    al = moe.moe_align(ids.to(dev), E, block_m)
    s, off, _ = ref.align(ids, E, block_m)
    rows = torch.full((len(s), H), 7.0, dtype=dtype, device=dev)
    got, at = moe.moe_permute(x.to(dev), ids.to(dev), al, weights=None if w is None else w.to(dev), rows=rows)
    assert got is rows
    assert torch.equal(at.cpu(), ref.pair_rows(ids, E, block_m))
    want = torch.full((len(s), H), 7.0, dtype=torch.float64)  # behind the last run: as it was
    want[:off[E]] = 0.0
    P = M * k
    for r, p in enumerate(s):
        if p < P:
            want[r] = x[p // k].double() * (1.0 if w is None else float(w.view(-1)[p]))
    if w is None:
        assert torch.equal(got.cpu().double(), want)
    else:
        close(got, want, want.abs() * (HALF[dtype] * 1.01 + U), "rows")


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("M,k,E,H,block_m,dtype", [(3000, 4, 16, 4096, 128, BF), (1500, 4, 16, 4104, 64, F32)])
def test_many_rows(dev, M, k, E, H, block_m, dtype, weighted):
    """Over 96 MB of rows, which go by tokens: padding, dropped pairs and rows behind
    the last run, and the gradients back."""
    import moe_layer_topk_amd as moe
    ids, x, w, g = make(M, k, E, H, dtype, weighted, True, 11)
    al = moe.moe_align(ids.to(dev), E, block_m)
    at = ref.pair_rows(ids, E, block_m)
    s, off, _ = ref.align(ids, E, block_m)
    assert len(s) * H * x.element_size() > 96 << 20
    rows = torch.full((len(s), H), 7.0, dtype=dtype, device=dev)
    wd = None if w is None else w.to(dev)
    _, got_at = moe.moe_permute(x.to(dev), ids.to(dev), al, weights=wd, rows=rows)
    assert torch.equal(got_at.cpu(), at)
    live = at.view(-1) >= 0
    held, owner = at.view(-1)[live].long(), torch.arange(M).repeat_interleave(k)[live]
    want = torch.full((len(s), H), 7.0, dtype=torch.float64)
    want[:off[E]] = 0.0
    want[held] = x.double()[owner] * (1.0 if w is None else w.double().view(-1)[live][:, None])
    close(rows, want, want.abs() * (HALF[dtype] * 1.01 + U) * (w is not None), "rows")
    src = torch.randn(len(s), H, generator=g).to(dtype)
    drows = torch.full_like(rows, 7.0)
    _, dw = moe.moe_unpermute_backward(x.to(dev), None if w is None else src.to(dev), wd, at.to(dev), al, drows=drows)
    assert torch.equal(drows, rows)  # the same product, w x
    if w is not None:
        prod = src.double()[held] * x.double()[owner]
        wdw, mag = torch.zeros(M * k, dtype=torch.float64), torch.zeros(M * k, dtype=torch.float64)
        wdw[live], mag[live] = prod.sum(1), prod.abs().sum(1)
        close(dw.view(-1), wdw, (H + 2) * U * mag, "dweights")


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("M,k,E,H,block_m,dtype,weighted", CASES)
def test_unpermute(dev, M, k, E, H, block_m, dtype, weighted, dropped):
    import moe_layer_topk_amd as moe
    ids, _, w, g = make(M, k, E, H, dtype, weighted, dropped, 2)
    at = ref.pair_rows(ids, E, block_m)
    s, _, _ = ref.align(ids, E, block_m)
    rows = torch.randn(len(s), H, generator=g).to(dtype)
    held = torch.zeros(len(s), dtype=torch.bool)
    held[at[at >= 0].long()] = True
    rows[~held] = float("nan")  # rows of no pair are not read into anything
    want, mag = ref.unpermute(rows, at, w)
    for odt in (dtype, F32 if dtype == BF else BF):
        out = moe.moe_unpermute(rows.to(dev), at.to(dev), weights=None if w is None else w.to(dev), out_dtype=odt)
        assert out.dtype == odt
        close(out, want, want.abs() * HALF[odt] + 2 * (k + 1) * U * mag, f"out {odt}")


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("M,k,E,H,block_m,dtype,weighted", CASES)
def test_unpermute_backward(dev, M, k, E, H, block_m, dtype, weighted, dropped):
    import moe_layer_topk_amd as moe
    ids, dout, w, g = make(M, k, E, H, dtype, weighted, dropped, 3)
    al = moe.moe_align(ids.to(dev), E, block_m)
    at = ref.pair_rows(ids, E, block_m)
    s, off, _ = ref.align(ids, E, block_m)
    rows = torch.randn(len(s), H, generator=g).to(dtype)
    drows = torch.full((len(s), H), 7.0, dtype=dtype, device=dev)
    dw_, wd = None, None if w is None else w.to(dev)
    moe.moe_unpermute_backward(dout.to(dev), None, wd, at.to(dev), al, drows=drows)
    if w is not None:
        again, dw_ = moe.moe_unpermute_backward(dout.to(dev), rows.to(dev), wd, at.to(dev), al,
                                                drows=torch.full_like(drows, 7.0))
        assert torch.equal(again, drows)
    want = torch.full((len(s), H), 7.0, dtype=torch.float64)
    want[:off[E]] = 0.0
    wdw = torch.zeros(M, k, dtype=torch.float64)
    mag = torch.zeros(M, k, dtype=torch.float64)
    for t in range(M):
        for j in range(k):
            r = int(at[t, j])
            if r >= 0:
                d = dout[t].double()
                want[r] = d * (1.0 if w is None else float(w[t, j]))
                wdw[t, j] = (d * rows[r].double()).sum()
                mag[t, j] = (d * rows[r].double()).abs().sum()
    close(drows, want, want.abs() * (HALF[dtype] * 1.01 + U), "drows")
    if w is not None:
        close(dw_, wdw, (H + 2) * U * mag, "dweights")


@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("M,k,E,H,block_m,dtype,weighted", CASES)
def test_permute_backward(dev, M, k, E, H, block_m, dtype, weighted, dropped):
    import moe_layer_topk_amd as moe
    ids, x, w, g = make(M, k, E, H, dtype, weighted, dropped, 4)
    at = ref.pair_rows(ids, E, block_m)
    s, _, _ = ref.align(ids, E, block_m)
    drows = torch.randn(len(s), H, generator=g).to(dtype)
    want, mag = ref.unpermute(drows, at, w)
    dx, dw_ = moe.moe_permute_backward(drows.to(dev), at.to(dev), None if w is None else x.to(dev),
                                       None if w is None else w.to(dev))
    close(dx, want, want.abs() * HALF[dtype] + 2 * (k + 1) * U * mag, "dx")
    if w is None:
        assert dw_ is None
        return
    live = at >= 0
    prod = drows.double()[at.clamp(min=0).long()] * x.double()[:, None, :] * live[:, :, None]
    close(dw_, prod.sum(2), (H + 2) * U * prod.abs().sum(2), "dweights")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pair_order(dev, dtype):
    """Without pair_row the rows are in pair order: moe_combine's bits, and its gradient."""
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(5)
    M, k, H = 37, 6, 1032
    y = torch.randn(M * k, H, generator=g).to(dtype).to(dev)
    w = torch.rand(M, k, generator=g).to(dev)
    assert torch.equal(moe.moe_unpermute(y, weights=w), moe.moe_combine(y, w, k))
    assert torch.equal(moe.moe_unpermute(y, topk=k), moe.moe_combine(y, torch.ones_like(w), k))
    at = torch.arange(M * k, dtype=torch.int32, device=dev).view(M, k)
    d = torch.randn(M, H, generator=g).to(dtype).to(dev)
    for a, b in zip(moe.moe_unpermute_backward(d, y, w), moe.moe_unpermute_backward(d, y, w, at)):
        assert torch.equal(a, b)
    for a, b in zip(moe.moe_permute_backward(y, None, d, w), moe.moe_permute_backward(y, at, d, w)):
        assert torch.equal(a, b)


def test_gradients_against_differences(dev):
    """The sum of dout * out is linear in the rows and in the weights, and so is the
    forward direction in x: differences of the calls themselves are exact but for
    the float32 sums (64 terms of size 1 a row, then H of them)."""
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(6)
    M, k, E, H, bm = 19, 4, 12, 264, 16
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32).to(dev)
    al = moe.moe_align(ids, E, bm)
    x, w = torch.randn(M, H, generator=g).to(dev), torch.rand(M, k, generator=g).to(dev)
    rows, at = moe.moe_permute(x, ids, al, weights=w)
    rows = torch.where(torch.isfinite(rows), rows, torch.zeros_like(rows))
    d = torch.randn(rows.shape, generator=g).to(dev)
    dx, dwp = moe.moe_permute_backward(d, at, x, w)

    def loss(x, w):
        r, a = moe.moe_permute(x, ids, al, weights=w, rows=torch.zeros_like(rows))
        return float((r.double() * d.double()).sum())

    vx, vw = torch.randn(M, H, generator=g).to(dev), torch.randn(M, k, generator=g).to(dev)
    tol = 1e-5 * float((rows.abs() * d.abs()).sum())
    assert abs(loss(x + vx, w) - loss(x - vx, w) - 2 * float((vx.double() * dx.double()).sum())) < 4 * tol
    assert abs(loss(x, w + vw) - loss(x, w - vw) - 2 * float((vw.double() * dwp.double()).sum())) < 4 * tol
    dout = torch.randn(M, H, generator=g).to(dev)
    drows, dwu = moe.moe_unpermute_backward(dout, rows, w, at, al)

    def back(r, w):
        return float((moe.moe_unpermute(r, at, w).double() * dout.double()).sum())

    vr = torch.randn(rows.shape, generator=g).to(dev)
    held = at.view(-1).long()
    want = 2 * float((vr.double()[held] * drows.double()[held]).sum())
    assert abs(back(rows + vr, w) - back(rows - vr, w) - want) < 4 * tol
    assert abs(back(rows, w + vw) - back(rows, w - vw) - 2 * float((vw.double() * dwu.double()).sum())) < 4 * tol


def test_in_place_and_repeat(dev):
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(7)
    M, k, E, H, bm = 200, 8, 16, 2048, 64
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32).to(dev)
    al = moe.moe_align(ids, E, bm)
    dout, w = torch.randn(M, H, generator=g).bfloat16().to(dev), torch.rand(M, k, generator=g).to(dev)
    rows, at = moe.moe_permute(dout, ids, al, weights=w, rows=torch.zeros(al["sorted_ids"].numel(), H, dtype=BF, device=dev))
    d1, w1 = moe.moe_unpermute_backward(dout, rows, w, at, al, drows=torch.zeros_like(rows))
    again = [moe.moe_unpermute_backward(dout, rows, w, at, al, drows=torch.zeros_like(rows)) for _ in range(3)]
    assert all(torch.equal(a, d1) and torch.equal(b, w1) for a, b in again)
    buf = rows.clone()
    d2, w2 = moe.moe_unpermute_backward(dout, buf, w, at, al, drows=buf)
    assert torch.equal(d1, d2) and torch.equal(w1, w2)


def test_empty_batch(dev):
    import moe_layer_topk_amd as moe
    ids = torch.empty(0, 2, dtype=torch.int32, device=dev)
    al = moe.moe_align(ids, 4, 16)
    rows, at = moe.moe_permute(torch.empty(0, 64, device=dev), ids, al)
    assert rows.shape == (0, 64) and at.shape == (0, 2)
    assert moe.moe_unpermute(rows, at).shape == (0, 64)
    assert moe.moe_permute_backward(rows, at)[0].shape == (0, 64)
    d, w = moe.moe_unpermute_backward(torch.empty(0, 64, device=dev), rows, torch.empty(0, 2, device=dev), at, al)
    assert d.shape == (0, 64) and w.shape == (0, 2)


def test_rows_no_call_wrote_are_not_followed(dev):
    """A pair_row outside the rows adds nothing and is written nowhere."""
    import moe_layer_topk_amd as moe
    rows = torch.ones(4, 64, device=dev)
    at = torch.tensor([[0, 4], [-1, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=dev)
    out = moe.moe_unpermute(rows, at)
    assert out[:, 0].tolist() == [1.0, 1.0, 0.0]
    drows = torch.zeros_like(rows)
    _, dw = moe.moe_unpermute_backward(2 * torch.ones(3, 64, device=dev), rows, torch.ones(3, 2, device=dev), at, drows=drows)
    assert drows[:, 0].tolist() == [2.0, 0.0, 0.0, 2.0]
    assert dw.tolist() == [[128.0, 0.0], [0.0, 128.0], [0.0, 0.0]]


def test_rows_past_four_gib(dev):
    """560,000 rows of 8 KB: every row comes back, offsets past 32 bits included."""
    import moe_layer_topk_amd as moe
    M, k, E, H = 70000, 8, 64, 4096
    g = torch.Generator(device=dev).manual_seed(8)
    ids = torch.randint(0, E, (M, k), generator=g, device=dev, dtype=torch.int32)
    al = moe.moe_align(ids, E, 1)
    x = torch.randint(-8, 9, (M, H), generator=g, device=dev).bfloat16()
    rows, at = moe.moe_permute(x, ids, al)
    assert rows.numel() * 2 > 2 ** 32
    for t in (0, 1, 34567, M - 1):
        assert torch.equal(rows[at[t].long()], x[t].expand(k, H))
    out, _ = moe.moe_permute_backward(rows, at)  # eight times a small integer: exact
    assert torch.equal(out, x * 8)
    d, dw = moe.moe_unpermute_backward(x, rows, torch.full((M, k), 0.5, device=dev), at, al, drows=rows)
    assert torch.equal(d[at[M - 1].long()], (x[M - 1] * 0.5).expand(k, H))
    assert torch.equal(dw[M - 1], (x[M - 1].float() ** 2).sum().expand(k))


def test_streams_and_graphs(dev):
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(9)
    M, k, E, H, bm = 50, 4, 8, 1024, 16
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32).to(dev)
    al = moe.moe_align(ids, E, bm)
    x, w = torch.randn(M, H, generator=g).to(dev), torch.rand(M, k, generator=g).to(dev)
    bufs = [torch.zeros(al["sorted_ids"].numel(), H, device=dev) for _ in range(2)]
    at = torch.empty(M, k, dtype=torch.int32, device=dev)
    out, dw = torch.empty(M, H, device=dev), torch.empty(M, k, device=dev)

    def step():
        moe.moe_permute(x, ids, al, weights=w, rows=bufs[0], pair_row=at)
        moe.moe_unpermute(bufs[0], at, weights=w, out=out)
        moe.moe_unpermute_backward(out, bufs[0], w, at, al, drows=bufs[1], dweights=dw)

    def results():
        return [t.clone() for t in (bufs[0], out, bufs[1], dw)]

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn(M, H, generator=g).to(dev) if i % 2 else x)
        out.zero_(), dw.zero_(), bufs[0].zero_(), bufs[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = results()
        out.zero_(), dw.zero_(), bufs[0].zero_(), bufs[1].zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, results()))
        if i == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_differences_to_the_sums_roundings(dev):
    """As above, from buffers that hold nothing but what was put there, each bound from
    the magnitudes S that meet in it: an operand moved by v (1 U), its product (1 U), on
    both sides; a sum over a token's k rows ((k + 1) U) or over a row's H terms
    ((H + 2) U), on both sides of a difference or once, against 2 v."""
    import moe_layer_topk_amd as moe
    g = torch.Generator().manual_seed(16)
    M, k, E, H, bm = 23, 4, 12, 264, 16
    ids = torch.randint(0, E, (M, k), generator=g, dtype=torch.int32).to(dev)
    al = moe.moe_align(ids, E, bm)

    def randn(*shape):
        return torch.randn(*shape, generator=g).to(dev)

    x, w, dout, vx, vw = randn(M, H), torch.rand(M, k, generator=g).to(dev), randn(M, H), randn(M, H), randn(M, k)
    empty = torch.zeros(al["sorted_ids"].numel(), H, device=dev)
    d, vr = randn(*empty.shape), randn(*empty.shape)
    rows, at = moe.moe_permute(x, ids, al, weights=w, rows=empty.clone())
    held = at.view(-1).long()

    def pairs(t):  # [M, k, H] of expert rows
        return t.double()[held].view(M, k, H)

    def tok(t):  # [M, 1, H] of token rows
        return t.double()[:, None, :]

    def wgt(t):  # [M, k, 1] of weights
        return t.double()[:, :, None]

    def check(lhs, rhs, terms, mags, what):
        bound = terms * U * float(mags.expand(M, k, H).sum())
        assert abs(float(lhs) - float(rhs)) <= bound, f"{what}: {float(lhs)} and {float(rhs)}, bound {bound}"

    def there(x, w):
        r, _ = moe.moe_permute(x, ids, al, weights=w, rows=empty.clone())
        return (r.double() * d.double()).sum()

    dx, dwp = moe.moe_permute_backward(d, at, x, w)
    check(there(x + vx, w) - there(x - vx, w), 2 * (vx.double() * dx.double()).sum(), 2 * k + 7,
          wgt(w).abs() * (tok(x).abs() + tok(vx).abs()) * pairs(d).abs(), "dx")
    check(there(x, w + vw) - there(x, w - vw), 2 * (vw.double() * dwp.double()).sum(), 2 * H + 9,
          (wgt(w).abs() + wgt(vw).abs()) * tok(x).abs() * pairs(d).abs(), "dweights of permute")

    def back(r, w):
        return (moe.moe_unpermute(r, at, w).double() * dout.double()).sum()

    drows, dwu = moe.moe_unpermute_backward(dout, rows, w, at, al, drows=empty.clone())
    check(back(rows + vr, w) - back(rows - vr, w), 2 * (pairs(vr) * pairs(drows)).sum(), 2 * k + 7,
          wgt(w).abs() * (pairs(rows).abs() + pairs(vr).abs()) * tok(dout).abs(), "drows")
    check(back(rows, w + vw) - back(rows, w - vw), 2 * (vw.double() * dwu.double()).sum(), 2 * H + 2 * k + 9,
          (wgt(w).abs() + wgt(vw).abs()) * pairs(rows).abs() * tok(dout).abs(), "dweights of unpermute")
