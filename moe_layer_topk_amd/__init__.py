"""Fused top-k Mixture-of-Experts layer for MI355X (gfx950).

A thin binding over libmoe.so: every function here only allocates output
tensors with torch, marshals pointers and calls the C entry point of the
same name on torch's current HIP stream.  All arithmetic runs in the HIP
kernels; there is no CPU or framework fallback (a missing library raises).

Steps of the layer (FusedMoE vs MegaMoE post, sections 2 and 3.1):
moe_route -> moe_align -> moe_grouped_gemm (gate/up + SiLU-and-mul, then
down) -> moe_combine, or all of them in one call with fused_moe.  For e4m3
weights the intermediate is float32 and the down call quantises it on load;
moe_quant_act gives the same codes as a tensor.  Block-scaled e4m3 (weights
float8_e4m3fn with float32 scales [E, N/128, K/128], one per 128 x 128 block;
[E] or [E, 1, 1] are one scale an expert): moe_quant_block
-> moe_grouped_gemm with the E4M3 kinds, or the fused layers from bfloat16
hidden states.  moe_route_grouped / fused_moe_grouped route with a Routing
(softmax or sigmoid scores, balance bias, expert groups).
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import (  # noqa: F401
    MOE_ERR_SCRATCH,
    MOE_ERR_UNSUPPORTED,
    MOE_W4A16,
    MOE_BF16,
    MOE_F32,
    MOE_FP8_BLOCK,
    MOE_FP8_E4M3,
    MOE_GEMM_DOWN,
    MOE_GEMM_DOWN_E4M3_ACT,
    MOE_GEMM_GATE_UP_SILU,
    MOE_GEMM_GATE_UP_SILU_E4M3,
    MOE_SCORE_SIGMOID,
    MOE_SCORE_SOFTMAX,
    AlignBufs,
    ExpertWeights,
    MoeError,
    RoutingArgs,
    check,
    lib,
)

# weight storage -> layer dtype (uint8 weights are packed int4 codes, W4A16)
_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_FP8_E4M3, torch.uint8: MOE_W4A16}
_INTER = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_FP8_E4M3: torch.bfloat16,
          MOE_W4A16: torch.bfloat16, MOE_FP8_BLOCK: torch.bfloat16}  # y and out
_ACT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_FP8_E4M3: torch.float32,
        MOE_W4A16: torch.bfloat16}  # the intermediate


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError("moe_layer_topk_amd computes on the GPU only; got a CPU tensor")
    # (the handle alone: 0.16 us a call, with torch's stream object 2.2)
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(t.device.index))


def moe_dtype(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def _layer_dtype(w: torch.Tensor, w_scale) -> int:
    """The layer dtype of expert weights: e4m3 with 3-D scales is block-scaled,
    unless they are one scale for each expert kept in three dimensions ([E, 1, 1]).
    The two meet only where one block is a whole matrix: block-scaled then, since
    matrices that small are no multiples of 256, as per-expert scales need."""
    if w.dtype == torch.float8_e4m3fn and w_scale is not None and w_scale.dim() == 3:
        E, N, K = w.shape
        if w_scale.numel() != E or w_scale.shape == (E, N // 128, K // 128):
            return MOE_FP8_BLOCK
    return moe_dtype(w)


def _call(fn, what: str, dev, *args) -> None:
    """fn(*args) with dev the current device (the library launches on it)."""
    if dev.index == torch.cuda.current_device():
        check(fn(*args), what)
    else:
        with torch.cuda.device(dev):
            check(fn(*args), what)


def _need(name: str, t, dtypes, shape, device) -> None:
    """A contiguous tensor of one of the dtypes, of this shape, on this device."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.is_contiguous()
            and t.device == device):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is missing")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} is not contiguous")


_F32, _F8 = (torch.float32,), (torch.float8_e4m3fn,)
_CODES = (torch.float8_e4m3fn, torch.uint8)


class Routing:
    """How a grouped router scores and chooses its experts (moe_routing in
    include/moe.h): score "softmax" or "sigmoid", a float32 bias [E] for the
    choice only (or None), n_groups groups of consecutive experts of which a
    token may use topk_groups, a group's score the best (group_top 1) or the
    sum of the two best (2) choices in it, renormalised weights, a factor."""

    _SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}

    def __init__(self, score: str = "softmax", bias=None, n_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                 renormalize: bool = True, scale: float = 1.0):
        if score not in self._SCORES:
            raise ValueError(f"score is one of {sorted(self._SCORES)}, got {score!r}")
        for name, v in (("n_groups", n_groups), ("topk_groups", topk_groups), ("group_top", group_top)):
            if not 0 <= v < 2 ** 31:  # (ctypes would take it modulo 2^32)
                raise ValueError(f"{name} is {v}")
        self.args = RoutingArgs(self._SCORES[score], None, n_groups, topk_groups, group_top, int(renormalize), scale)
        self._ref = ctypes.byref(self.args)
        self.bias = bias

    @property
    def bias(self):
        """The balance bias.  A program may change its values in place or set
        another tensor; calls made after that use it.  A captured call goes on
        reading the tensor it was captured with, which has to live as long."""
        return self._bias

    @bias.setter
    def bias(self, bias) -> None:
        if bias is not None:
            if not bias.is_cuda:
                raise ValueError("moe_layer_topk_amd computes on the GPU only; got a CPU bias")
            _need("bias", bias, _F32, (bias.numel(),), bias.device)
        self._bias = bias  # kept alive: the calls read it
        self._at = self.args.bias = None if bias is None else bias.data_ptr()

    def _check(self, E: int, device) -> None:
        # (at each call: a tensor's storage may have moved since it was set; the few
        # comparisons here are 0.4 us of a one-token call's 7, the checks below 0.8)
        b = self._bias
        if b is not None and (b.data_ptr() != self._at or b.numel() != E or b.device != device or not b.is_contiguous()):
            _need("bias", b, _F32, (E,), device)
            self._at = self.args.bias = b.data_ptr()


def moe_route_grouped(logits: torch.Tensor, topk: int, routing: Routing, topk_ids=None, topk_weights=None):
    """Top-k ids (int32 [M,k]) and weights (float32 [M,k]) of a grouped router
    from float32 or bfloat16 logits [M,E]."""
    M, E = logits.shape
    dev = logits.device
    stream = _stream(logits)
    _need("logits", logits, (torch.float32, torch.bfloat16), (M, E), dev)
    routing._check(E, dev)
    if topk_ids is None:
        topk_ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
    _need("topk_ids", topk_ids, (torch.int32,), (M, topk), dev)
    _need("topk_weights", topk_weights, _F32, (M, topk), dev)
    _call(lib().moe_route_grouped, "moe_route_grouped", dev, _DTYPES[logits.dtype], logits.data_ptr(), routing._ref, M, E,
          topk, topk_ids.data_ptr(), topk_weights.data_ptr(), stream)
    return topk_ids, topk_weights


def moe_route(logits: torch.Tensor, topk: int, renormalize: bool = True, topk_ids=None, topk_weights=None):
    """Top-k ids (int32 [M,k]) and weights (float32 [M,k]) from float32 logits [M,E]."""
    M, E = logits.shape
    ids = topk_ids if topk_ids is not None else torch.empty((M, topk), dtype=torch.int32, device=logits.device)
    wts = topk_weights if topk_weights is not None else torch.empty((M, topk), dtype=torch.float32,
                                                                    device=logits.device)
    check(lib().moe_route(_p(logits), M, E, topk, int(renormalize), _p(ids), _p(wts), _stream(logits)),
          "moe_route")
    return ids, wts


def moe_align_capacity(M: int, topk: int, E: int, block_m: int) -> int:
    return lib().moe_align_capacity(M, topk, E, block_m)


def moe_align(topk_ids: torch.Tensor, E: int, block_m: int) -> dict:
    """Index system of the sorted pairs (see moe_align_bufs in include/moe.h)."""
    M, topk = topk_ids.shape
    cap = moe_align_capacity(M, topk, E, block_m)
    dev = topk_ids.device
    i32 = dict(dtype=torch.int32, device=dev)
    out = {
        "sorted_ids": torch.empty(max(cap, 1), **i32),
        "tile_expert": torch.empty(max(cap // block_m, 1), **i32),
        "expert_counts": torch.empty(E, **i32),
        "expert_offsets": torch.empty(E + 1, **i32),
        "active_experts": torch.empty(max(min(E, M * topk), 1), **i32),
        "num_active": torch.empty(1, **i32),
        "block_m": block_m,
        "pairs": M * topk,
    }
    check(lib().moe_align(_p(topk_ids), M, topk, E, block_m, align_struct(out), _stream(topk_ids)), "moe_align")
    return out


def align_struct(al: dict) -> AlignBufs:
    return AlignBufs(*(al[n].data_ptr() for n in
                       ("sorted_ids", "tile_expert", "expert_counts", "expert_offsets", "active_experts",
                        "num_active")))


def moe_grouped_gemm(kind: int, a: torch.Tensor, w: torch.Tensor, al: dict, M: int, topk: int,
                     a_scale=None, w_scale=None, c=None, c_amax=None):
    """GATE_UP: act[P, N/2] = silu(gate) * up;  DOWN: y[P, N].  Returns (c, c_amax)."""
    E, N, K = w.shape
    dt = _layer_dtype(w, w_scale)
    if dt == MOE_FP8_BLOCK:
        return _block_gemm(kind, a, w, al, M, topk, a_scale, w_scale, c, c_amax)
    if dt == MOE_W4A16:
        K *= 2  # two 4-bit codes per byte
    P = M * topk
    cols = N // 2 if kind == MOE_GEMM_GATE_UP_SILU else N
    if kind != MOE_GEMM_GATE_UP_SILU and (kind == MOE_GEMM_DOWN_E4M3_ACT) != (a.dtype == torch.float8_e4m3fn):
        raise ValueError("MOE_GEMM_DOWN_E4M3_ACT takes e4m3 act codes and e4m3 weights; DOWN takes the act")
    if kind != MOE_GEMM_GATE_UP_SILU and kind != MOE_GEMM_DOWN_E4M3_ACT and a.dtype != _ACT[dt]:
        raise ValueError(f"DOWN with {w.dtype} weights takes a {_ACT[dt]} intermediate, got {a.dtype}")
    if c is None:
        c = torch.empty((P, cols), dtype=_ACT[dt] if kind == MOE_GEMM_GATE_UP_SILU else _INTER[dt], device=w.device)
    if dt == MOE_FP8_E4M3 and kind == MOE_GEMM_GATE_UP_SILU and c_amax is None:
        c_amax = torch.empty(1, dtype=torch.float32, device=w.device)
    bufs = align_struct(al)
    check(lib().moe_grouped_gemm(kind, dt, _p(a), _p(a_scale), _p(w), _p(w_scale), ctypes.byref(bufs), M, topk,
                                 E, N, K, al["block_m"], _p(c), _p(c_amax), _stream(w)), "moe_grouped_gemm")
    return c, c_amax


def _block_gemm(kind, a, w, al, M, topk, a_scale, w_scale, c, c_scale):
    """moe_grouped_gemm on block-scaled e4m3 weights; returns (c, scales of c or None)."""
    E, N, K = w.shape
    P, dev = M * topk, w.device
    stream = _stream(w)
    gate = kind in (MOE_GEMM_GATE_UP_SILU, MOE_GEMM_GATE_UP_SILU_E4M3)
    codes = kind in (MOE_GEMM_GATE_UP_SILU_E4M3, MOE_GEMM_DOWN_E4M3_ACT)
    rows, cols = (M, N // 2) if gate else (P, N)
    _need("w", w, _F8, (E, N, K), dev)
    _need("w_scale", w_scale, _F32, (E, N // 128, K // 128), dev)
    if kind == MOE_GEMM_DOWN:
        _need("a", a, _F32, (rows, K), dev)
    else:
        _need("a", a, _CODES, (rows, K), dev)
        _need("a_scale", a_scale, _F32, (rows, K // 128), dev)
    cdt = torch.bfloat16 if not gate else torch.float8_e4m3fn if codes else torch.float32
    if c is None:
        c = torch.empty((P, cols), dtype=cdt, device=dev)
    _need("c", c, _CODES if gate and codes else (cdt,), (P, cols), dev)
    if kind == MOE_GEMM_GATE_UP_SILU_E4M3:
        if c_scale is None:
            c_scale = torch.empty((P, cols // 128), dtype=torch.float32, device=dev)
        _need("c_amax (the scales of c)", c_scale, _F32, (P, cols // 128), dev)
    block_m = al["block_m"]
    if al["pairs"] != P or al["expert_counts"].numel() != E or al["sorted_ids"].device != dev:
        raise ValueError("the alignment (moe_align) is of another batch, number of experts or device")
    bufs = align_struct(al)
    _call(lib().moe_grouped_gemm, "moe_grouped_gemm", dev, kind, MOE_FP8_BLOCK, _p(a), _p(a_scale), _p(w), _p(w_scale),
          ctypes.byref(bufs), M, topk, E, N, K, block_m, _p(c), _p(c_scale), stream)
    return c, c_scale


def moe_quant_block(x: torch.Tensor, block_rows: int = 1, q=None, scale=None):
    """Block-scaled e4m3 of x [rows, K] (float32 or bfloat16): (codes float8_e4m3fn
    [rows, K], float32 scales [ceil(rows / block_rows), K / 128]); block_rows 1
    for token rows, 128 for weights."""
    rows, K = x.shape
    dev = x.device
    stream = _stream(x)
    _need("x", x, (torch.float32, torch.bfloat16), (rows, K), dev)
    if block_rows < 1:
        raise ValueError("block_rows is 1 or 128")
    shape = (-(-rows // block_rows), K // 128)
    if q is None:
        q = torch.empty((rows, K), dtype=torch.float8_e4m3fn, device=dev)
    if scale is None:
        scale = torch.empty(shape, dtype=torch.float32, device=dev)
    _need("q", q, _CODES, (rows, K), dev)
    _need("scale", scale, _F32, shape, dev)
    _call(lib().moe_quant_block, "moe_quant_block", dev, _DTYPES[x.dtype], x.data_ptr(), rows, K, block_rows, q.data_ptr(),
          scale.data_ptr(), stream)
    return q, scale


def moe_quant_act(act: torch.Tensor, amax: torch.Tensor, out=None):
    """e4m3 codes (torch.float8_e4m3fn, same shape) of the float32 intermediate with scale amax/448."""
    if act.dtype != torch.float32:
        raise ValueError("moe_quant_act takes the float32 intermediate")
    q = out if out is not None else torch.empty(act.shape, dtype=torch.float8_e4m3fn, device=act.device)
    check(lib().moe_quant_act(_p(act), _p(amax), act.numel(), _p(q), _stream(act)), "moe_quant_act")
    return q


def moe_combine(y: torch.Tensor, topk_weights: torch.Tensor, topk: int, out_dtype=None, out=None):
    P, H = y.shape
    M = P // topk
    odt = y.dtype if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((M, H), dtype=odt, device=y.device)
    check(lib().moe_combine(moe_dtype(y), _p(y), _p(topk_weights), M, topk, H, moe_dtype(out), _p(out),
                            _stream(y)), "moe_combine")
    return out


def moe_block_m(dtype: int, M: int, E: int, topk: int) -> int:
    """Rows per tile (block_m) the fused layer aligns such a batch to; 0 for invalid arguments."""
    return lib().moe_block_m(dtype, M, E, topk)


def fused_moe_workspace_size(dtype: int, M: int, E: int, topk: int, H: int, I: int) -> int:
    return lib().fused_moe_workspace_size(dtype, M, E, topk, H, I)


def _check_block_weights(w1, w2, w1_scale, w2_scale, dev) -> None:
    """The experts of a layer on block-scaled e4m3 weights."""
    E, twoI, H = w1.shape
    I = twoI // 2
    _need("w1", w1, _F8, (E, 2 * I, H), dev)
    _need("w2", w2, _F8, (E, H, I), dev)
    _need("w1_scale", w1_scale, _F32, (E, 2 * I // 128, H // 128), dev)
    _need("w2_scale", w2_scale, _F32, (E, H // 128, I // 128), dev)


def _check_layer(dt: int, x, w1, w2, x_scale, w1_scale, w2_scale, dev) -> None:
    """x and the experts of a layer of any dtype (scales of a dtype that has none
    are left for the library to refuse)."""
    M, H = x.shape
    E, I = w1.shape[0], w1.shape[1] // 2
    if dt == MOE_FP8_BLOCK:
        _check_block_weights(w1, w2, w1_scale, w2_scale, dev)
        _need("x", x, (torch.bfloat16,), (M, w1.shape[2]), dev)
        return
    per_byte = 2 if dt == MOE_W4A16 else 1  # weights in an element
    _need("w1", w1, (w1.dtype,), (E, 2 * I, H // per_byte), dev)
    _need("w2", w2, (w1.dtype,), (E, H, I // per_byte), dev)
    xdt = {MOE_W4A16: (torch.bfloat16,), MOE_FP8_E4M3: _CODES}.get(dt, (w1.dtype,))
    _need("x", x, xdt, (M, H), dev)
    if dt == MOE_W4A16:
        _need("w1_scale", w1_scale, _F32, (E, H // 128, 2 * I), dev)
        _need("w2_scale", w2_scale, _F32, (E, I // 128, H), dev)
    elif dt == MOE_FP8_E4M3:  # one number for each expert (x: one), in any shape
        for name, t, n in (("x_scale", x_scale, 1), ("w1_scale", w1_scale, E), ("w2_scale", w2_scale, E)):
            _need(name, t, _F32, t.shape if t is not None and t.numel() == n else (n,), dev)


def _check_batch(dt: int, x, logits, E: int, topk: int, out, topk_ids, topk_weights, workspace, dev) -> None:
    """What a call brings beside x and the weights (workspace None: the library's own)."""
    M = x.shape[0]
    _need("router_logits", logits, _F32, (M, E), dev)
    _need("out", out, (_INTER[dt],), (M, x.shape[1]), dev)
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != dev):
        raise ValueError(f"the workspace is {workspace.dtype} on {workspace.device}, expected torch.uint8 on {dev}")
    if workspace is not None and not workspace.is_contiguous():  # (its bytes are counted from its first)
        raise ValueError("the workspace is not contiguous")
    if topk_ids is not None:
        _need("topk_ids", topk_ids, (torch.int32,), (M, topk), dev)
    if topk_weights is not None:
        _need("topk_weights", topk_weights, _F32, (M, topk), dev)


def _layer_call(dt: int, what: str, dev, *args) -> None:
    """The layer function `what`; a block-scaled layer on its tensors' device."""
    if dt == MOE_FP8_BLOCK:
        _call(getattr(lib(), what), what, dev, *args)
    else:
        check(getattr(lib(), what)(*args), what)


def fused_moe_grouped(x, router_logits, w1, w2, topk: int, routing: Routing, x_scale=None, w1_scale=None,
                      w2_scale=None, workspace=None, out=None, topk_ids=None, topk_weights=None):
    """The whole layer with a grouped router (float32 logits); returns out[M,H]
    (float32 for fp32 weights, bfloat16 otherwise)."""
    M, H = x.shape
    E, twoI, _ = w1.shape
    I = twoI // 2
    dev = x.device
    stream = _stream(x)
    dt = _layer_dtype(w1, w1_scale)
    _check_layer(dt, x, w1, w2, x_scale, w1_scale, w2_scale, dev)
    routing._check(E, dev)
    if workspace is None:
        need = fused_moe_workspace_size(dt, M, E, topk, H, I)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((M, H), dtype=_INTER[dt], device=dev)
    _check_batch(dt, x, router_logits, E, topk, out, topk_ids, topk_weights, workspace, dev)
    _call(lib().fused_moe_grouped, "fused_moe_grouped", dev, dt, _p(x), _p(x_scale), _p(router_logits), routing._ref,
          _p(w1), _p(w1_scale), _p(w2), _p(w2_scale), M, E, topk, H, I, _p(out), _p(topk_ids), _p(topk_weights),
          _p(workspace), workspace.numel(), stream)
    return out


def fused_moe(x, router_logits, w1, w2, topk: int, renormalize: bool = True, x_scale=None, w1_scale=None,
              w2_scale=None, workspace=None, out=None, topk_ids=None, topk_weights=None):
    """The whole layer; returns out[M,H] (float32 for fp32 weights, bfloat16 otherwise)."""
    M, H = x.shape
    E, twoI, _ = w1.shape
    I = twoI // 2
    dt = _layer_dtype(w1, w1_scale)
    need = fused_moe_workspace_size(dt, M, E, topk, H, I)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, H), dtype=_INTER[dt], device=x.device)
    if dt == MOE_FP8_BLOCK:
        _check_block_weights(w1, w2, w1_scale, w2_scale, x.device)
        _need("x", x, (torch.bfloat16,), (M, w1.shape[2]), x.device)
        _check_batch(dt, x, router_logits, E, topk, out, topk_ids, topk_weights, workspace, x.device)
    _layer_call(dt, "fused_moe", x.device, dt, _p(x), _p(x_scale), _p(router_logits), _p(w1), _p(w1_scale), _p(w2),
                _p(w2_scale), M, E, topk, H, I, int(renormalize), _p(out), _p(topk_ids), _p(topk_weights),
                _p(workspace), workspace.numel(), _stream(x))
    return out


def fused_moe_noalloc(x, router_logits, w1, w2, topk: int, renormalize: bool = True, x_scale=None, w1_scale=None,
                      w2_scale=None, out=None, topk_ids=None, topk_weights=None):
    """fused_moe with the library's static device scratch as its workspace
    (no workspace argument; calls overlapping on one GPU race)."""
    M, H = x.shape
    E, twoI, _ = w1.shape
    I = twoI // 2
    dt = _layer_dtype(w1, w1_scale)
    if out is None:
        out = torch.empty((M, H), dtype=_INTER[dt], device=x.device)
    if dt == MOE_FP8_BLOCK:
        _check_block_weights(w1, w2, w1_scale, w2_scale, x.device)
        _need("x", x, (torch.bfloat16,), (M, w1.shape[2]), x.device)
        _check_batch(dt, x, router_logits, E, topk, out, topk_ids, topk_weights, None, x.device)
    _layer_call(dt, "fused_moe_noalloc", x.device, dt, _p(x), _p(x_scale), _p(router_logits), _p(w1), _p(w1_scale),
                _p(w2), _p(w2_scale), M, E, topk, H, I, int(renormalize), _p(out), _p(topk_ids), _p(topk_weights),
                _stream(x))
    return out


def moe_router_logits(x, router_w, x_scale=None, out=None):
    """Router scores float32 [M, E] = x . router_w^T (router_w float32 [E, H])."""
    M, H = x.shape
    E = router_w.shape[0]
    if router_w.dtype != torch.float32:
        raise ValueError("router weights are float32")
    lg = out if out is not None else torch.empty((M, E), dtype=torch.float32, device=x.device)
    check(lib().moe_router_logits(moe_dtype(x), _p(x), _p(x_scale), _p(router_w), M, H, E, _p(lg), _stream(x)),
          "moe_router_logits")
    return lg


def fused_moe_router(x, router_w, w1, w2, topk: int, renormalize: bool = True, x_scale=None, w1_scale=None,
                     w2_scale=None, workspace=None, out=None, logits=None, topk_ids=None, topk_weights=None):
    """The whole layer from the hidden states: router scores on the GPU (written
    to `logits`, float32 [M, E]), then route -> align -> experts -> combine.
    Returns (out, logits)."""
    M, H = x.shape
    E, twoI, _ = w1.shape
    I = twoI // 2
    dt = _layer_dtype(w1, w1_scale)
    need = fused_moe_workspace_size(dt, M, E, topk, H, I)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, H), dtype=_INTER[dt], device=x.device)
    if logits is None:
        logits = torch.empty((M, E), dtype=torch.float32, device=x.device)
    if dt == MOE_FP8_BLOCK:
        _check_block_weights(w1, w2, w1_scale, w2_scale, x.device)
        _need("x", x, (torch.bfloat16,), (M, w1.shape[2]), x.device)
        _check_batch(dt, x, logits, E, topk, out, topk_ids, topk_weights, workspace, x.device)
        _need("router_w", router_w, _F32, (E, H), x.device)
    _layer_call(dt, "fused_moe_router", x.device, dt, _p(x), _p(x_scale), _p(router_w), _p(logits), _p(w1), _p(w1_scale),
                _p(w2), _p(w2_scale), M, E, topk, H, I, int(renormalize), _p(out), _p(topk_ids), _p(topk_weights),
                _p(workspace), workspace.numel(), _stream(x))
    return out, logits


class ExpertCache:
    """Expert streaming (the MoE inference post, FusedMoE vs MegaMoE, sections
    4.1-4.3): the experts' weights stay in pinned host memory and a GPU pool of
    `capacity` slots holds the ones in use.  Calling the cache runs the layer
    (fused_moe_cached): route, copy in the missing experts (least recently
    used slot first), then the fused layer over the slots.  prefetch() copies
    experts ahead of a call on the cache's own copy stream.

    w1, w2 (and the scales of fp8 or W4A16 weights) are the layer's weights
    in fused_moe's layout, on the host; they are copied once into pinned
    memory unless already pinned."""

    def __init__(self, w1, w2, capacity: int, w1_scale=None, w2_scale=None, device=None, copy_stream=None):
        self.dtype = _layer_dtype(w1, w1_scale)
        self.E, twoI = w1.shape[0], w1.shape[1]
        self.I, self.H, self.capacity = twoI // 2, w2.shape[1], capacity
        device = torch.device("cuda" if device is None else device)
        self.device = device if device.index is not None else torch.device("cuda", torch.cuda.current_device())
        parts = (w1, w2, w1_scale, w2_scale)
        if any(t is not None and t.is_cuda for t in parts):
            raise ValueError("ExpertCache takes the experts' weights on the host")
        if self.dtype == MOE_FP8_BLOCK:
            _check_block_weights(*(t if t is None else t.contiguous() for t in parts), w1.device)
        self.host = [None if t is None else (t.contiguous() if t.is_pinned() else t.contiguous().pin_memory())
                     for t in parts]
        self.slots = [None if t is None else torch.empty((capacity,) + tuple(t.shape[1:]), dtype=t.dtype,
                                                         device=self.device) for t in parts]
        # default priority: copies overlap compute through events, not priorities
        self.copy_stream = copy_stream if copy_stream is not None else torch.cuda.Stream(self.device)
        self._host_ids = torch.empty(0, dtype=torch.int32, pin_memory=True)
        self._ws = None
        h = ctypes.c_void_p()
        check(lib().moe_cache_create(self.dtype, self.E, self.H, self.I, capacity, ExpertWeights(*map(_p, self.host)),
                                     ExpertWeights(*map(_p, self.slots)), ctypes.c_void_p(self.copy_stream.cuda_stream),
                                     ctypes.byref(h)), "moe_cache_create")
        self._h = h

    def prefetch(self, experts) -> None:
        ids = torch.as_tensor(list(experts), dtype=torch.int32)
        check(lib().moe_cache_prefetch(self._h, _p(ids), ids.numel()), "moe_cache_prefetch")

    def stats(self) -> dict:
        v = [ctypes.c_int64() for _ in range(4)]
        check(lib().moe_cache_stats(self._h, *map(ctypes.byref, v)), "moe_cache_stats")
        return dict(zip(("hits", "misses", "prefetched", "h2d_bytes"), (x.value for x in v)))

    def __call__(self, x, router_logits, topk: int, renormalize: bool = True, x_scale=None, workspace=None,
                 out=None, topk_ids=None, topk_weights=None):
        """The layer over the cache; returns out[M,H] as fused_moe does."""
        M = x.shape[0]
        if self._host_ids.numel() < M * topk:
            # the previous call's copy from the old buffer may still be queued
            torch.cuda.current_stream(x.device).synchronize()
            self._host_ids = torch.empty(M * topk, dtype=torch.int32, pin_memory=True)
        if workspace is None:
            need = max(fused_moe_workspace_size(self.dtype, M, self.capacity, topk, self.H, self.I), 1)
            if self._ws is None or self._ws.numel() < need:
                self._ws = torch.empty(need, dtype=torch.uint8, device=x.device)
            workspace = self._ws
        if out is None:
            out = torch.empty((M, self.H), dtype=_INTER[self.dtype], device=x.device)
        if self.dtype == MOE_FP8_BLOCK:
            _need("x", x, (torch.bfloat16,), (M, self.H), self.device)
            _check_batch(self.dtype, x, router_logits, self.E, topk, out, topk_ids, topk_weights, workspace, self.device)
        _layer_call(self.dtype, "fused_moe_cached", self.device, self._h, _p(x), _p(x_scale), _p(router_logits), M, topk,
                    int(renormalize), _p(out), _p(topk_ids), _p(topk_weights), _p(self._host_ids), _p(workspace),
                    workspace.numel(), _stream(x))
        return out

    def close(self) -> None:
        if getattr(self, "_h", None):
            check(lib().moe_cache_destroy(self._h), "moe_cache_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
