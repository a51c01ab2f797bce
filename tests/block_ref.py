"""Plain float64 forms (torch on the CPU) of the grouped router and of the
block-scaled e4m3 operators, for the tests.  Nothing here is shared with the
library."""
import math

import torch

FP8_MAX = 448.0
TINY = 2.0 ** -126


def route(logits, topk, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    """(ids int32, weights float64) token by token, as include/moe.h defines them."""
    M, E = logits.shape
    gs = E // n_groups
    ids = torch.empty(M, topk, dtype=torch.int32)
    wts = torch.empty(M, topk, dtype=torch.float64)
    b = [0.0] * E if bias is None else [float(v) for v in bias.double()]
    for t in range(M):
        row = [float(v) if v == v else -math.inf for v in logits[t].double().tolist()]
        if score == "sigmoid":
            s = [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in row]
        else:
            m = max(row)
            ex = [0.0 if m == -math.inf else 1.0 if v == m else math.exp(v - m) for v in row]
            den = math.fsum(ex)
            s = [v / den if den > 0 else 0.0 for v in ex]
        c = [x + y for x, y in zip(s, b)]
        c = [-math.inf if v != v else v for v in c]
        rank = row if bias is None else c
        left = list(range(E))
        if topk_groups < n_groups:
            group = []
            for g in range(n_groups):
                top = sorted(c[g * gs:(g + 1) * gs], reverse=True)[:group_top]
                v = sum(top)
                group.append(-math.inf if v != v else v)
            keep = sorted(range(n_groups), key=lambda g: (-group[g], g))[:topk_groups]
            left = [e for e in range(E) if e // gs in keep]
        sel = sorted(left, key=lambda e: (-rank[e], e))[:topk]
        w = [s[e] for e in sel]
        if renormalize:
            den = math.fsum(w)
            w = [v / den if den > 0 else 0.0 for v in w]
        ids[t] = torch.tensor(sel, dtype=torch.int32)
        wts[t] = torch.tensor(w, dtype=torch.float64) * scale
    return ids, wts


def quant(x, block_rows):
    """(codes float8_e4m3fn, scales float32): IEEE float32 quotients on the CPU."""
    x = x.float()
    n, K = x.shape
    nb = -(-n // block_rows)
    p = torch.cat([x, x.new_zeros(nb * block_rows - n, K)]).view(nb, block_rows, K // 128, 128)
    amax = p.abs().amax((1, 3))
    s = torch.maximum(amax / torch.tensor(FP8_MAX), torch.tensor(TINY))
    q = (p / s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    bad = ~torch.isfinite(amax)
    s[bad] = math.nan
    v = q.view(torch.uint8)
    v[bad[:, None, :, None].expand_as(v)] = 0x7F
    return v.view(nb * block_rows, K)[:n].view(torch.float8_e4m3fn), s


def value(q, s, block_rows):
    n, K = q.shape
    nb = s.shape[0]
    v = torch.zeros(nb * block_rows, K, dtype=torch.float64)
    v[:n] = q.float().double()
    return (v.view(nb, block_rows, K // 128, 128) * s.double()[:, None, :, None]).view(-1, K)[:n]


def products(a, w, ids, topk, gate):
    """(c, bound) of the grouped GEMM in float64: a [rows][K] values, w [E][N][K]
    values, ids [M][topk].  bound: how far the kernels' sums may be from c.

    The products of two e4m3 values are exact in float32; a block's 128 are
    summed in an order the hardware picks and the K/128 sums after that, each
    addition off by at most one step (2^-23) of the magnitudes added so far,
    and the scales' product and its use round twice more.  DOWN runs on the
    f8f6f4 MFMA, which keeps the bits of eight consecutive products down to
    2^-13 of the largest one's power of two: each of the eight may lose less
    than that, 2^-10 of the largest in all."""
    P, (E, N, K) = ids.numel(), w.shape
    c = torch.zeros(P, N, dtype=torch.float64)
    mag = torch.zeros(P, N, dtype=torch.float64)
    cut = torch.zeros(P, N, dtype=torch.float64)
    for p, e in enumerate(ids.reshape(-1).tolist()):
        row = a[p // topk if gate else p]
        prod = w[e] * row
        c[p] = prod.sum(1)
        mag[p] = prod.abs().sum(1)
        if not gate:
            cut[p] = prod.abs().view(N, K // 8, 8).amax(2).sum(1)
    return c, mag * (128 + K // 128 + 2) * 2.0 ** -23 + cut * 2.0 ** -10


def silu_mul(h, bound):
    """act = silu(g) u and its bound: |silu'| <= 1.1, and a few roundings of the
    exponential (its argument's rounding grows with |g|), the quotient and the product."""
    I = h.shape[1] // 2
    g, u, dg, du = h[:, :I], h[:, I:], bound[:, :I], bound[:, I:]
    s = g * torch.sigmoid(g)
    act = s * u
    return act, 1.1 * dg * u.abs() + s.abs() * du + dg * du * 1.1 + act.abs() * (8 + 2 * g.abs()) * 2.0 ** -24
