"""Grouped router on the GPU against the float64 form in block_ref.

Ids must be equal.  Weights: float32 exponentials (about 2 half-steps each, and
one for every unit of |l - l_max| their argument's rounding costs), a sum whose
terms are positive, a quotient and a product: (32 + span) half-steps of 2^-24,
span the row's largest finite |l - l_max|, at most 104 (past that a float32
exponential is 0 and so is the weight).
"""
import math

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


def check(dev, logits, topk, bias=None, **kw):
    import moe_layer_topk_amd as moe
    r = moe.Routing(bias=None if bias is None else bias.to(dev), **kw)
    ids, wts = moe.moe_route_grouped(logits.to(dev), topk, r)
    torch.cuda.synchronize()
    rid, rw = ref.route(logits, topk, bias=bias, **kw)
    assert torch.equal(ids.cpu(), rid), (ids.cpu() != rid).any(1).nonzero().flatten()[:8]
    f = logits.double()
    fin = torch.where(torch.isfinite(f), f, torch.zeros_like(f))
    span = (fin.amax(1, keepdim=True) - fin.amin(1, keepdim=True)).clamp_max(104.0)
    assert torch.isfinite(wts).all()
    err = (wts.cpu().double() - rw).abs()
    assert bool((err <= (32 + span) * 2.0 ** -24 * rw.abs() + 1e-37).all()), float(err.max())
    return ids, wts


def draw(M, E, seed, dtype=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, E, generator=g) * spread).to(dtype), torch.randn(E, generator=g) * 0.05


SHAPES = [(1, 256, 8, 8, 4), (3, 256, 8, 8, 4), (300, 256, 8, 8, 4), (17, 160, 6, 8, 3), (65, 128, 8, 1, 1),
          (5, 8, 2, 1, 1), (9, 8, 4, 4, 2), (130, 200, 8, 5, 2), (33, 64, 16, 4, 1), (2, 255, 16, 5, 3), (4, 1, 1, 1, 1),
          (6, 3, 3, 1, 1), (7, 256, 16, 64, 8), (64, 96, 1, 16, 16), (1000, 40, 6, 4, 3)]


@pytest.mark.parametrize("M,E,k,G,T", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
def test_route(dev, M, E, k, G, T, score, top, biased):
    if top > E // G:
        pytest.skip("a group holds one expert")
    print(f"route M={M} E={E} k={k} G={G} T={T} {score} top={top} bias={biased}", flush=True)
    lg, b = draw(M, E, M * 7 + E)
    check(dev, lg, k, bias=b if biased else None, score=score, n_groups=G, topk_groups=T, group_top=top,
          renormalize=(M + k) % 2 == 0, scale=2.5 if M % 2 else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bf16_ties(dev, score):
    """bfloat16 logits tie often; biases on a coarse grid tie the choices too."""
    lg, b = draw(500, 128, 3, torch.bfloat16)
    lg = (lg.float() * 4).round().div(4).to(torch.bfloat16)
    check(dev, lg, 8, score=score, n_groups=8, topk_groups=4, group_top=2)
    check(dev, lg, 8, bias=(b * 40).round() / 4, score=score, n_groups=8, topk_groups=4, group_top=2)
    check(dev, torch.zeros(5, 256), 8, bias=torch.zeros(256), score=score, n_groups=8, topk_groups=2, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_close_choices(dev, score):
    """Choices closer than float32 can tell apart: float64 decides."""
    g = torch.Generator().manual_seed(11)
    E = 64
    lg = torch.randn(40, E, generator=g)
    for t in range(40):  # experts in pairs whose logits differ by a few steps
        lg[t, 1::2] = torch.nextafter(lg[t, 0::2], torch.full((E // 2,), math.inf if t % 2 else -math.inf))
    check(dev, lg, 8, bias=torch.zeros(E), score=score)
    check(dev, lg, 8, bias=torch.full((E,), 64.0), score=score, n_groups=8, topk_groups=3, group_top=2)
    # a bias that cancels the scores' difference up to rounding
    b = -torch.sigmoid(lg[0].double()).float()
    check(dev, lg[:1].clone(), 8, bias=b, score="sigmoid", n_groups=4, topk_groups=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_infinities_and_nan(dev, score, biased):
    inf, nan = math.inf, math.nan
    lg, b = draw(12, 64, 5)
    lg[0] = -inf                       # nothing left
    lg[1, 3:] = -inf                   # fewer experts than slots
    lg[2, 5] = nan
    lg[3] = nan
    lg[4, 7] = inf
    lg[5, 9] = inf
    lg[5, 50] = inf
    lg[6] = torch.finfo(torch.float32).min
    lg[7, ::2] = torch.finfo(torch.float32).min
    lg[8] = 1e30
    lg[9, 1:] = -200.0                 # scores that underflow in float32
    lg[10, :32] = -inf                 # whole groups masked
    for kw in (dict(), dict(n_groups=8, topk_groups=2, group_top=2), dict(n_groups=8, topk_groups=8, group_top=1)):
        check(dev, lg, 8, bias=b if biased else None, score=score, **kw)
    b2 = b.clone()
    b2[4], b2[5], b2[6] = inf, -inf, nan
    check(dev, lg, 8, bias=b2, score=score, n_groups=8, topk_groups=3, group_top=2)


def test_route_into_given_buffers_on_a_side_stream(dev):
    import moe_layer_topk_amd as moe
    lg, b = draw(70, 256, 9)
    r = moe.Routing("sigmoid", b.to(dev), 8, 4, 2, True, 2.5)
    x = lg.to(dev)
    ids = torch.full((72, 8), -7, dtype=torch.int32, device=dev)
    w = torch.full((72, 8), -7.0, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.moe_route_grouped(x, 8, r, topk_ids=ids[:70], topk_weights=w[:70])
    s.synchronize()
    rid, _ = ref.route(lg, 8, "sigmoid", b, 8, 4, 2, True, 2.5)
    assert torch.equal(ids[:70].cpu(), rid)
    assert bool((ids[70:] == -7).all()) and bool((w[70:] == -7.0).all())  # rows past the batch stay
