"""Float64 forms of what stands around the experts (rows in expert order, norms
around a block, gradients of the experts' products), for tests."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step of a rounding, relative
U = 2.0 ** -24  # half a step of a float32 operation


def align(ids, E, block_m):
    """(sorted pair ids, offsets [E + 1], counts) of ids [M, k], as moe_align makes them."""
    flat = ids.reshape(-1).tolist()
    P = len(flat)
    cap = -(-(P + min(E, P) * (block_m - 1)) // block_m) * block_m
    out, offsets, counts = [], [0], []
    for e in range(E):
        run = [p for p, i in enumerate(flat) if i == e]
        counts.append(len(run))
        out += run + [P] * (-len(run) % block_m)
        offsets.append(len(out))
    return out + [P] * (cap - len(out)), offsets, counts


def pair_rows(ids, E, block_m):
    """The row of every pair (-1 without an expert), [M, k]."""
    s, _, _ = align(ids, E, block_m)
    at = np.full(ids.numel(), -1, np.int32)
    for r, p in enumerate(s):
        if p < ids.numel():
            at[p] = r
    return torch.from_numpy(at).view(ids.shape)


def unpermute(rows, at, w):
    """(sum, sum of magnitudes) over a token's pairs, float64."""
    M, k = at.shape
    live = (at >= 0) & (at < rows.shape[0])
    v = torch.where(live[:, :, None], rows.double()[at.clamp(0, rows.shape[0] - 1).long()], torch.zeros((), dtype=torch.float64))
    if w is not None:
        v = v * torch.where(live, w.double(), torch.zeros((), dtype=torch.float64))[:, :, None]
    return v.sum(1), v.abs().sum(1)


def rms_norm(v, eps):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def residual_norm(h, y, post, gate, scale, pre, eps):
    out = h
    if y is not None:
        u = y if post is None else rms_norm(y, eps) * post
        out = h + scale * (u if gate is None else u * gate)
    return out, None if pre is None else rms_norm(out, eps) * pre


def silu_mul(z):
    I = z.shape[1] // 2
    return z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]


def close(got, want, bound, what):
    """Every element within its own bound (float64 tensors on the CPU)."""
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound) & ~(got == want) & ~(torch.isnan(got) & torch.isnan(want))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i]} for {want[i]}, bound "
                             f"{bound[i] if isinstance(bound, torch.Tensor) else bound}")
