"""The grouped router on every number of experts a lane, group layout and logit
type together, against the float64 form (bounds as in test_gpu_route_grouped)."""
import math

import pytest
import torch

from test_gpu_route_grouped import check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_layer_topk_amd as moe
    moe.lib()
    return torch.device("cuda:0")


# (tokens, experts, topk, groups, groups kept).  One expert a lane (up to 64), two
# (up to 128) or four; groups of whole lanes (a power of two of them) or not;
# numbers of experts that whole vectors of a lane do and do not divide
SHAPES = [(50, 96, 8, 8, 3), (50, 120, 6, 5, 2), (50, 128, 8, 8, 3), (50, 127, 8, 1, 1), (50, 99, 4, 9, 4), (50, 256, 8, 8, 4),
          (50, 200, 8, 5, 2), (50, 255, 16, 5, 3), (50, 40, 6, 4, 3), (50, 64, 8, 4, 2), (50, 63, 8, 7, 3), (1, 7, 3, 1, 1)]


@pytest.mark.parametrize("M,E,k,G,T", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_shapes(dev, M, E, k, G, T, dtype, score, biased):
    print(f"M={M} E={E} k={k} G={G} T={T} {dtype} {score} bias={biased}", flush=True)
    for top in (1, 2):
        lg, b = draw(M, E, M + E + top, dtype)
        check(dev, lg, k, bias=b if biased else None, score=score, n_groups=G, topk_groups=T, group_top=top,
              renormalize=top == 1, scale=2.5 if biased else 1.0)


# inputs whose choices float32 seldom settles: wide logits, experts disabled by
# their bias, biases of another size than the scores
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [1.0, 6.0, 30.0])
@pytest.mark.parametrize("off", [None, -math.inf, -1e9, -1e4, -20.0])
def test_wide_logits_and_disabled_experts(dev, score, spread, off):
    lg, b = draw(200, 256, 4, spread=spread)
    if off is not None:
        b[17] = off
        b[200:203] = off
    check(dev, lg, 8, bias=b, score=score, n_groups=8, topk_groups=4, group_top=2, scale=2.5)
    check(dev, lg, 8, bias=b, score=score)
    if off is not None:
        check(dev, lg, 8, bias=torch.where(b == off, b, torch.zeros_like(b)), score=score, n_groups=8, topk_groups=4, group_top=2)
