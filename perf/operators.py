"""Cases of the block-scaled e4m3 experts and the grouped router, for timing.

Five operators, as a program that serves such a layer calls them:

  route    top-k routing on softmax or sigmoid scores, with a bias for balance
           that only the choice sees, groups of experts, renormalised weights
  quant    e4m3 codes with one float32 scale per 128 values of a row (tokens)
           or per 128 x 128 block (weights)
  gate_up  the experts' gate/up product over routed rows on codes and scales,
           SiLU-and-mul, and the intermediate as codes and scales again
  down     the experts' down product on those, bfloat16 rows out
  layer    all of it from bfloat16 hidden states: route, quantise, align,
           gate/up, down, weighted combine

`own` false: each in its plain form (elementary torch operations in float32,
float64 where a choice or a rounding hangs on it).  `own` true: the calls a
user makes of moe_layer_topk_amd.
"""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
TINY = 2.0 ** -126  # a block of zeros takes the smallest normal scale


# ------------------------------------------------------------------- cases

def listed():
    grp = dict(score="sigmoid", bias=True, n_groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5)
    flat = dict(score="softmax", bias=False, n_groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0)
    return [
        # one decode token through a grouped sigmoid router: latency alone
        dict(name="route_grouped_1", op="route", M=1, E=256, topk=8, logits="f32", **grp),
        # a long prefill batch through the same router
        dict(name="route_grouped_16384", op="route", M=16384, E=256, topk=8, logits="f32", **grp),
        # fine-grained experts, plain softmax of bfloat16 scores, an odd batch
        dict(name="route_softmax_2049", op="route", M=2049, E=128, topk=8, logits="bf16", **flat),
        # the hidden states of a small decode batch
        dict(name="quant_tokens_5", op="quant", rows=5, K=4096, block_rows=1, dtype="bf16"),
        # the float32 intermediate of a prefill batch
        dict(name="quant_rows_4096", op="quant", rows=4096, K=14336, block_rows=1, dtype="f32"),
        # decode batch over many wide experts: a few rows each, bound by the weights' stream
        dict(name="gate_up_decode_32", op="gate_up", M=32, E=64, topk=8, H=4096, I=8192, skew=False),
        # wide experts, prefill with skewed routing: bound by the matrix cores
        dict(name="gate_up_prefill_4096", op="gate_up", M=4096, E=8, topk=2, H=4096, I=14336, skew=True),
        # wide experts, the largest decode batch
        dict(name="down_decode_64", op="down", M=64, E=8, topk=2, H=4096, I=14336, skew=False),
        # fine-grained prefill, ragged rows per expert
        dict(name="down_prefill_2048", op="down", M=2048, E=128, topk=8, H=2048, I=768, skew=False),
        # one token through the whole fine-grained layer
        dict(name="layer_decode_1", op="layer", M=1, E=128, topk=8, H=2048, I=768, skew=False, **grp),
        # an odd decode batch of wide experts
        dict(name="layer_decode_77", op="layer", M=77, E=8, topk=2, H=4096, I=14336, skew=False, **flat),
        # fine-grained prefill through the whole layer
        dict(name="layer_prefill_4096", op="layer", M=4096, E=128, topk=8, H=2048, I=768, skew=False, **grp),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_routing(rng, E, topk):
    """A router for E experts: flat, or groups that leave at least topk experts."""
    score = rng.choice(["softmax", "sigmoid"])
    fits = [(g, t) for g in (1, 2, 4, 5, 8, 16) if E % g == 0 and E // g >= 2
            for t in range(1, g + 1) if t * (E // g) >= topk]
    g, t = rng.choice(fits)
    return dict(score=score, bias=rng.random() < 0.6, n_groups=g, topk_groups=t, group_top=rng.choice([1, 2]),
                renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))


def draw(rng):
    """One more case of the same ranges; never more work than the largest listed."""
    most = [work(c) for c in listed()]
    top = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["route", "quant", "gate_up", "down", "layer"])
        E = rng.choice([8, 16, 40, 64, 96, 128, 160, 200, 256])
        topk = rng.choice([1, 2, 4, 6, 8])
        if op == "route":
            c = dict(op=op, M=_log_int(rng, 1, 16384), E=E, topk=topk, logits=rng.choice(["f32", "bf16"]),
                     **_draw_routing(rng, E, topk))
        elif op == "quant":
            c = dict(op=op, rows=_log_int(rng, 1, 8192), K=BLOCK * _log_int(rng, 2, 112),
                     block_rows=rng.choice([1, 1, 128]), dtype=rng.choice(["bf16", "f32"]))
        else:
            c = dict(op=op, M=_log_int(rng, 1, 4096), E=E, topk=topk, H=BLOCK * _log_int(rng, 2, 56),
                     I=BLOCK * _log_int(rng, 1, 112), skew=rng.random() < 0.3)
            if op == "layer":
                c.update(_draw_routing(rng, E, topk))
            if 3 * c["E"] * c["H"] * c["I"] > 1.5e9:
                continue
        w = work(c)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return c


def work(case):
    """Bytes and operations one pass cannot do without."""
    c = case
    if c["op"] == "route":
        b = 4 if c["logits"] == "f32" else 2
        return {"bytes": c["M"] * c["E"] * b + 8 * c["M"] * c["topk"] + 4 * c["E"], "flops": 4 * c["M"] * c["E"]}
    if c["op"] == "quant":
        n = c["rows"] * c["K"]
        b = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * (b + 1) + 4 * -(-c["rows"] // c["block_rows"]) * (c["K"] // BLOCK), "flops": 2 * n}
    M, E, k, H, I = c["M"], c["E"], c["topk"], c["H"], c["I"]
    P = M * k
    active = min(E * (1.0 - (1.0 - k / E) ** M), P)  # experts that M tokens reach, routed evenly
    sc = 1.0 + 4.0 / BLOCK  # a code and its share of a row's scale
    if c["op"] == "gate_up":
        return {"bytes": active * 2 * I * H + M * H * sc + P * I * sc, "flops": 4.0 * P * H * I}
    if c["op"] == "down":
        return {"bytes": active * I * H + P * I * sc + P * H * 2, "flops": 2.0 * P * H * I}
    return {"bytes": active * 3 * I * H + 4 * M * H + 4 * M * E + 8 * P, "flops": 6.0 * P * H * I}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _round_blocks(v, rows):
    """e4m3 codes and float32 scales of a float32 matrix, one scale for each
    rows x 128 block: s = max(amax / 448, the smallest normal), code = v / s."""
    n, K = v.shape
    nb = -(-n // rows)
    p = v if nb * rows == n else torch.cat([v, v.new_zeros(nb * rows - n, K)])
    b = p.view(nb, rows, K // BLOCK, BLOCK)
    amax = b.abs().amax((1, 3))
    s = torch.clamp_min(amax / torch.full_like(amax, FP8_MAX), TINY)  # (a scalar divisor would round as a product)
    q = (b / s[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return q.view(nb * rows, K)[:n], s


def _expert_weights(g, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(E, N // BLOCK, K // BLOCK, device="cuda")
    for e in range(E):
        w[e], s[e] = _round_blocks(_normal(g, N, K) * 0.02, BLOCK)
    return w, s


def _logits(g, c):
    z = _normal(g, c["M"], c["E"])
    if c.get("skew"):
        p = torch.arange(1, c["E"] + 1, device="cuda", dtype=torch.float32) ** -1.1
        z = z + (p / p.sum()).log()
    return z


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] in ("route", "layer"):
        z = _logits(g, c)
        st["logits"] = z.bfloat16() if c.get("logits") == "bf16" else z
        # balance biases stay small next to the scores' own spread
        st["bias"] = _normal(g, c["E"]) * (0.05 if c["score"] == "sigmoid" else 0.002) if c["bias"] else None
    if c["op"] == "quant":
        v = _normal(g, c["rows"], c["K"])
        v *= torch.exp(_normal(g, c["rows"], 1))  # rows of different size
        st["x"] = v.bfloat16() if c["dtype"] == "bf16" else v
    if c["op"] in ("gate_up", "layer"):
        st["w1"], st["w1_s"] = _expert_weights(g, c["E"], 2 * c["I"], c["H"])
    if c["op"] in ("down", "layer"):
        st["w2"], st["w2_s"] = _expert_weights(g, c["E"], c["H"], c["I"])
    if c["op"] == "layer":
        st["x"] = _normal(g, c["M"], c["H"]).bfloat16()
    if c["op"] in ("gate_up", "down"):
        # routed rows: distinct experts for each token, and the list of every expert's pairs
        ids = torch.topk(_logits(g, c), c["topk"], dim=1).indices
        st["ids"] = ids.to(torch.int32)
        st["rows"] = _rows_of(ids, c["E"])
        n, K = (c["M"], c["H"]) if c["op"] == "gate_up" else (c["M"] * c["topk"], c["I"])
        v = _normal(g, n, K)
        st["a"], st["a_s"] = _round_blocks(v if c["op"] == "gate_up" else v * torch.sigmoid(v), 1)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """What a program keeps beside its inputs: output buffers, the router's
    description, the alignment of the routed rows, the layer's workspace."""
    import moe_layer_topk_amd as moe
    c = st["case"]
    dev = "cuda"
    if c["op"] in ("route", "layer"):
        st["routing"] = moe.Routing(score=c["score"], bias=st["bias"], n_groups=c["n_groups"],
                                    topk_groups=c["topk_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                                    scale=c["scale"])
        st["ids"] = torch.empty(c["M"], c["topk"], dtype=torch.int32, device=dev)
        st["wts"] = torch.empty(c["M"], c["topk"], device=dev)
    if c["op"] == "quant":
        st["q"] = torch.empty(c["rows"], c["K"], dtype=torch.float8_e4m3fn, device=dev)
        st["s"] = torch.empty(-(-c["rows"] // c["block_rows"]), c["K"] // BLOCK, device=dev)
    if c["op"] in ("gate_up", "down"):
        P = c["M"] * c["topk"]
        st["al"] = moe.moe_align(st["ids"], c["E"], moe.moe_block_m(moe.MOE_FP8_BLOCK, c["M"], c["E"], c["topk"]))
        if c["op"] == "gate_up":
            st["c"] = torch.empty(P, c["I"], dtype=torch.float8_e4m3fn, device=dev)
            st["c_s"] = torch.empty(P, c["I"] // BLOCK, device=dev)
        else:
            st["c"] = torch.empty(P, c["H"], dtype=torch.bfloat16, device=dev)
    if c["op"] == "layer":
        n = moe.fused_moe_workspace_size(moe.MOE_FP8_BLOCK, c["M"], c["E"], c["topk"], c["H"], c["I"])
        st["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
        st["out"] = torch.empty(c["M"], c["H"], dtype=torch.bfloat16, device=dev)


def _rows_of(ids, E):
    """Pair numbers of every expert, in order."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    n = torch.bincount(flat, minlength=E).tolist()
    return list(torch.split(order, n))


# --------------------------------------------------------------------- run

def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def _run_own(st):
    import moe_layer_topk_amd as moe
    c = st["case"]
    if c["op"] == "route":
        return moe.moe_route_grouped(st["logits"], c["topk"], st["routing"], topk_ids=st["ids"],
                                     topk_weights=st["wts"])
    if c["op"] == "quant":
        q, s = moe.moe_quant_block(st["x"], c["block_rows"], q=st["q"], scale=st["s"])
        return q.bfloat16(), s
    if c["op"] == "gate_up":
        q, s = moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP_SILU_E4M3, st["a"], st["w1"], st["al"], c["M"], c["topk"],
                                    a_scale=st["a_s"], w_scale=st["w1_s"], c=st["c"], c_amax=st["c_s"])
        return q.bfloat16(), s
    if c["op"] == "down":
        return moe.moe_grouped_gemm(moe.MOE_GEMM_DOWN_E4M3_ACT, st["a"], st["w2"], st["al"], c["M"], c["topk"],
                                    a_scale=st["a_s"], w_scale=st["w2_s"], c=st["c"])[0]
    out = moe.fused_moe_grouped(st["x"], st["logits"], st["w1"], st["w2"], c["topk"], st["routing"],
                                w1_scale=st["w1_s"], w2_scale=st["w2_s"], workspace=st["ws"], out=st["out"],
                                topk_ids=st["ids"], topk_weights=st["wts"])
    return out, st["ids"], st["wts"]


def _deq(q, s, rows):
    """float32 values of codes with one scale for each rows x 128 block."""
    v = q.float()
    n, K = v.shape
    return (v.view(-1, rows, K // BLOCK, BLOCK) * s[:, None, :, None]).view(n, K)


def _plain_route(st):
    c = st["case"]
    z = st["logits"].double()
    M, E = z.shape
    G = c["n_groups"]
    score = torch.softmax(z, 1) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-z))
    choice = score if st["bias"] is None else score + st["bias"].double()
    rank = z if st["bias"] is None else choice  # both scores rise with the logit
    if c["topk_groups"] < G:
        best = torch.sort(choice.view(M, G, E // G), dim=2, descending=True).values
        group = best[:, :, :c["group_top"]].sum(2)
        keep = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        live = torch.zeros(M, G, dtype=torch.bool, device=z.device).scatter_(1, keep, True)
        rank = rank.masked_fill(~live.repeat_interleave(E // G, 1), -math.inf)
    ids = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _plain_quant(st):
    c = st["case"]
    q, s = _round_blocks(st["x"].float(), c["block_rows"])
    return q.bfloat16(), s


def _gate_up(a, a_s, w, w_s, rows, topk, P):
    x = _deq(a, a_s, 1)
    I = w.shape[1] // 2
    act = torch.zeros(P, I, device=a.device)
    for e, p in enumerate(rows):
        if p.numel():
            h = x[p // topk] @ _deq(w[e], w_s[e], BLOCK).t()
            act[p] = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
    return _round_blocks(act, 1)


def _down(a, a_s, w, w_s, rows):
    x = _deq(a, a_s, 1)
    y = torch.zeros(x.shape[0], w.shape[1], device=a.device)
    for e, p in enumerate(rows):
        if p.numel():
            y[p] = x[p] @ _deq(w[e], w_s[e], BLOCK).t()
    return y


def _plain_gate_up(st):
    c = st["case"]
    q, s = _gate_up(st["a"], st["a_s"], st["w1"], st["w1_s"], st["rows"], c["topk"], c["M"] * c["topk"])
    return q.bfloat16(), s


def _plain_down(st):
    return _down(st["a"], st["a_s"], st["w2"], st["w2_s"], st["rows"]).bfloat16()


def _plain_layer(st):
    c = st["case"]
    ids, wts = _plain_route(st)
    x, x_s = _round_blocks(st["x"].float(), 1)
    rows = _rows_of(ids, c["E"])
    q, s = _gate_up(x, x_s, st["w1"], st["w1_s"], rows, c["topk"], c["M"] * c["topk"])
    y = _down(q, s, st["w2"], st["w2_s"], rows).view(c["M"], c["topk"], c["H"])
    return (y * wts[:, :, None]).sum(1).bfloat16(), ids, wts


_PLAIN = {"route": _plain_route, "quant": _plain_quant, "gate_up": _plain_gate_up, "down": _plain_down,
          "layer": _plain_layer}


# ------------------------------------------------------------------- exact
# The definitions in float64, written apart from the plain form above.

def _e4m3(v):
    """Nearest e4m3 value, ties to even: 3 mantissa bits down to 2^-6, then
    steps of 2^-9; magnitudes end at 448."""
    e = torch.frexp(v).exponent - 1  # 2^e <= |v| < 2^(e + 1)
    step = torch.exp2(e.clamp_min(-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _f32(v):
    """The nearest float32 values, held in float64: the operator's scales and
    quotients are float32 by definition (a tie of v / s between two codes is
    decided by the scale's rounding)."""
    return v.float().double()


def _exact_blocks(v, rows):
    """(values of the codes, scales) of a float64 matrix of float32 values."""
    n, K = v.shape
    if rows == 1:
        b = v.view(n, K // BLOCK, BLOCK)
        scale = _f32(b.abs().amax(2) / FP8_MAX).clamp_min(TINY)
        return _e4m3(_f32(b / scale[:, :, None])).view(n, K), scale
    codes = torch.empty_like(v)
    scale = v.new_empty(-(-n // rows), K // BLOCK)
    for i in range(scale.shape[0]):
        b = v[i * rows:(i + 1) * rows].reshape(-1, K // BLOCK, BLOCK)
        scale[i] = _f32(b.abs().amax((0, 2)) / FP8_MAX).clamp_min(TINY)
        codes[i * rows:(i + 1) * rows] = _e4m3(_f32(b / scale[i][None, :, None])).reshape(-1, K)
    return codes, scale


def _exact_route(st):
    c = st["case"]
    z = st["logits"].double()
    M, E, G = c["M"], c["E"], c["n_groups"]
    if c["score"] == "sigmoid":
        score = torch.sigmoid(z)
    else:
        ex = torch.exp(z - z.amax(1, keepdim=True))
        score = ex / ex.sum(1, keepdim=True)
    choice = score + (0.0 if st["bias"] is None else st["bias"].double())

    def take(v, n):
        """The n largest of each row, one after another, lowest index first among equals."""
        v, at = v.clone(), torch.arange(v.shape[1], device=v.device)
        got = []
        for _ in range(n):
            top = v.amax(1, keepdim=True)
            i = torch.where(v == top, at, v.shape[1]).amin(1, keepdim=True)
            got.append(i)
            v.scatter_(1, i, -math.inf)
        return torch.cat(got, 1)

    rank = (z if st["bias"] is None else choice).clone()
    if c["topk_groups"] < G:
        parts = choice.reshape(M * G, E // G)
        group = parts.gather(1, take(parts, c["group_top"])).sum(1).view(M, G)
        out = torch.ones(M, G, dtype=torch.bool, device=z.device)
        out.scatter_(1, take(group, c["topk_groups"]), False)
        rank.view(M, G, E // G)[out] = -math.inf
    ids = take(rank, c["topk"])
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w * c["scale"]


def _exact_value(q, s, rows):
    n, K = q.shape
    return (q.double().reshape(-1, rows, K // BLOCK, BLOCK) * s.double()[:, None, :, None]).reshape(n, K)


def _exact_gate_up(x, w1, w1_s, rows, topk, P):
    I = w1.shape[1] // 2
    act = torch.zeros(P, I, dtype=torch.float64, device=x.device)
    for e, p in enumerate(rows):
        if p.numel():
            w = _exact_value(w1[e], w1_s[e], BLOCK)
            t = x[p // topk]
            act[p] = torch.nn.functional.silu(t @ w[:I].t()) * (t @ w[I:].t())
    return _exact_blocks(_f32(act), 1)


def _exact_down(a, w2, w2_s, rows):
    y = torch.zeros(a.shape[0], w2.shape[1], dtype=torch.float64, device=a.device)
    for e, p in enumerate(rows):
        if p.numel():
            y[p] = a[p] @ _exact_value(w2[e], w2_s[e], BLOCK).t()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "route":
        return _exact_route(st)
    if c["op"] == "quant":
        return _exact_blocks(st["x"].double(), c["block_rows"])
    if c["op"] == "gate_up":
        return _exact_gate_up(_exact_value(st["a"], st["a_s"], 1), st["w1"], st["w1_s"], st["rows"], c["topk"],
                              c["M"] * c["topk"])
    if c["op"] == "down":
        return _exact_down(_exact_value(st["a"], st["a_s"], 1), st["w2"], st["w2_s"], st["rows"])
    ids, wts = _exact_route(st)
    rows = _rows_of(ids, c["E"])
    x, x_s = _exact_blocks(st["x"].double(), 1)
    q, s = _exact_gate_up(_exact_value(x, x_s, 1), st["w1"], st["w1_s"], rows, c["topk"], c["M"] * c["topk"])
    y = _exact_down(_exact_value(q, s, 1), st["w2"], st["w2_s"], rows).view(c["M"], c["topk"], c["H"])
    return (y * wts[:, :, None]).sum(1), ids, wts
