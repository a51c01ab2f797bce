"""Cases of what stands around the experts of a block that trains, for timing.

Three groups of operators, as a program that runs or trains such a block calls
them:

  permute, unpermute,        token rows brought into expert order and back, with the
  unpermute_backward         routing weights applied, and the gradients of the rows
                             and the weights
  norm, norm_backward        the norm after a block, its gate and residual scale, the
                             residual sum and the norm before the next block in one
                             pass, and the gradients of all of it
  gate_up, dx, dw            the experts' products as training needs them: gate and up
                             before SiLU-and-mul, the gradients of the rows (through
                             SiLU-and-mul, or plain) and of the weights

`own` false: each in its plain form (elementary torch operations in float32).
`own` true: the calls a user makes of moe_layer_topk_amd.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    wide = dict(E=8, topk=2, H=4096, I=14336)       # few wide experts
    fine = dict(E=128, topk=8, H=2048, I=768)       # many small ones
    return [
        # one decode token's rows for eight of 128 experts: latency alone
        dict(name="permute_1", op="permute", M=1, E=128, topk=8, H=2048, block_m=16, dtype="bf16", weighted=False,
             skew=False),
        # a prefill batch put into expert order without padding, as for sending rows to the experts' owners
        dict(name="permute_4096", op="permute", M=4096, E=128, topk=8, H=2048, block_m=1, dtype="bf16", weighted=False,
             skew=False),
        # an odd batch's expert rows back into token order with the routing weights
        dict(name="unpermute_2049", op="unpermute", M=2049, E=128, topk=8, H=2048, block_m=64, dtype="bf16",
             weighted=True, skew=False),
        # training batch of wide experts, skewed routing: gradients of expert rows and routing weights
        dict(name="unpermute_backward_4096", op="unpermute_backward", M=4096, E=8, topk=2, H=4096, block_m=128,
             dtype="bf16", weighted=True, skew=True),
        # one decode token between two blocks: latency alone
        dict(name="norm_1", op="norm", M=1, H=4096, dtype="bf16", block=True, post=True, gate="channel", pre=True),
        # a long prefill batch between two blocks, a gate for every token
        dict(name="norm_16384", op="norm", M=16384, H=4096, dtype="bf16", block=True, post=True, gate="token", pre=True),
        # the same place in a training step: gradients of the block, the stream, the weights and the gate
        dict(name="norm_backward_4096", op="norm_backward", M=4096, H=4096, dtype="bf16", block=True, post=True,
             gate="channel", pre=True),
        # gate and up kept for a backward pass, fine-grained training batch, ragged rows per expert
        dict(name="gate_up_2049", op="gate_up", M=2049, skew=False, **fine),
        # gradient through the down product and SiLU-and-mul, wide experts, skewed: bound by the matrix cores
        dict(name="dx_down_4096", op="dx", through="down", M=4096, skew=True, **wide),
        # gradient of a small batch's hidden states: bound by the weights' stream
        dict(name="dx_gate_up_16", op="dx", through="gate_up", M=16, skew=False, **fine),
        # weight gradients of wide experts, skewed: bound by the matrix cores
        dict(name="dw_gate_up_4096", op="dw", through="gate_up", M=4096, skew=True, out="bf16", **wide),
        # weight gradients of many small experts in float32: bound by their stores
        dict(name="dw_down_1023", op="dw", through="down", M=1023, skew=False, out="f32", **fine),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges; never more work than the largest listed."""
    most = [work(c) for c in listed()]
    top = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["permute", "unpermute", "unpermute_backward", "norm", "norm_backward", "gate_up", "dx", "dw"])
        if op in ("norm", "norm_backward"):
            block = rng.random() < 0.8
            pre = rng.random() < 0.8 or not block
            c = dict(op=op, M=_log_int(rng, 1, 16384), H=8 * _log_int(rng, 8, 2048), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     block=block, post=block and rng.random() < 0.7,
                     gate=rng.choice(["none", "channel", "token"]) if block else "none", pre=pre)
        else:
            E = rng.choice([4, 8, 16, 40, 64, 96, 128, 160, 256])
            c = dict(op=op, M=_log_int(rng, 1, 4096), E=E, topk=min(E, rng.choice([1, 2, 4, 6, 8])),
                     skew=rng.random() < 0.3)
            if op in ("gate_up", "dx", "dw"):
                c.update(H=128 * _log_int(rng, 2, 48), I=128 * _log_int(rng, 1, 112))
                if 2 * E * c["H"] * c["I"] > 1.0e9:
                    continue
                if op != "gate_up":
                    c["through"] = rng.choice(["down", "gate_up"])
                if op == "dw":
                    c["out"] = rng.choice(["bf16", "f32"])
            else:
                c.update(H=8 * _log_int(rng, 8, 1024), block_m=rng.choice([1, 16, 64, 128]),
                         dtype=rng.choice(["bf16", "bf16", "f32"]),
                         weighted=op == "unpermute_backward" or rng.random() < 0.6)
        w = work(c)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return c


def _size(name):
    return 4 if name == "f32" else 2


def work(case):
    """Bytes and operations one pass cannot do without."""
    c = case
    M, H = c["M"], c["H"]
    if c["op"] in ("norm", "norm_backward"):
        row = M * H * _size(c["dtype"])
        if c["op"] == "norm":
            n = (2 if c["block"] else 1) + (1 if c["block"] else 0) + (1 if c["pre"] else 0)
        else:  # y, h', the gradients of h' and x in; of y and h out
            n = 2 + (1 if c["pre"] else 0) + ((2 if c["block"] else 0) + 1)
        return {"bytes": n * row, "flops": 8 * n * M * H}
    P = M * c["topk"]
    if "I" not in c:
        b = _size(c["dtype"])
        n = {"permute": M + P, "unpermute": M + P, "unpermute_backward": M + 2 * P}[c["op"]]
        return {"bytes": n * H * b + 8 * P, "flops": 2 * P * H * (2 if c["op"] == "unpermute_backward" else 1)}
    E, I = c["E"], c["I"]
    active = min(E * (1.0 - (1.0 - c["topk"] / E) ** M), P)  # experts that M tokens reach, routed evenly
    if c["op"] == "gate_up":
        return {"bytes": 2 * (active * 2 * I * H + M * H + 2 * P * I), "flops": 4.0 * P * H * I}
    if c["op"] == "dx":
        if c["through"] == "down":  # dy, W2, gate and up in; their gradients and the activations out
            return {"bytes": 2 * (active * I * H + P * H + 5 * P * I), "flops": 2.0 * P * H * I}
        return {"bytes": 2 * (active * 2 * I * H + 2 * P * I + P * H), "flops": 4.0 * P * H * I}
    if c["through"] == "down":
        return {"bytes": E * H * I * _size(c["out"]) + 2 * P * (H + I), "flops": 2.0 * P * H * I}
    return {"bytes": E * 2 * I * H * _size(c["out"]) + 2 * (P * 2 * I + M * H), "flops": 4.0 * P * H * I}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(g, c):
    z = _normal(g, c["M"], c["E"])
    if c["skew"]:
        p = torch.arange(1, c["E"] + 1, device="cuda", dtype=torch.float32) ** -1.1
        z = z + (p / p.sum()).log()
    return z


def _alignment(ids, E, block_m):
    """The index system of routed pairs, as an alignment call of the framework
    leaves it: pairs sorted by expert, every expert's run padded with the number
    of pairs to a multiple of block_m."""
    M, k = ids.shape
    P = M * k
    i32 = dict(dtype=torch.int32, device=ids.device)
    cap = -(-(P + min(E, P) * (block_m - 1)) // block_m) * block_m
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    runs = (counts + block_m - 1) // block_m * block_m
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(runs, 0)
    first = torch.cumsum(counts, 0) - counts
    place = offsets[flat[order]] + torch.arange(P, device=ids.device) - first[flat[order]]
    sorted_ids = torch.full((cap,), P, **i32)
    sorted_ids[place] = order.int()
    tile_expert = torch.full((cap // block_m,), -1, **i32)
    tiles = torch.repeat_interleave(torch.arange(E, device=ids.device), runs // block_m)
    tile_expert[:tiles.numel()] = tiles.int()
    active = torch.full((min(E, P),), -1, **i32)
    live = counts.nonzero().flatten()
    active[:live.numel()] = live.int()
    return {"sorted_ids": sorted_ids, "tile_expert": tile_expert, "expert_counts": counts.int(),
            "expert_offsets": offsets.int(), "active_experts": active,
            "num_active": torch.tensor([live.numel()], **i32), "block_m": block_m, "pairs": P}


def _tile_rows(c):
    """Rows of a tile for the products: the taller where experts have many rows."""
    return 128 if c["M"] * c["topk"] > 48 * c["E"] else 64


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    M, H = c["M"], c["H"]
    dt = TYPES[c.get("dtype", "bf16")]

    def rows(n, cols, size=1.0):
        return (_normal(g, n, cols) * size).to(dt)

    if c["op"] in ("norm", "norm_backward"):
        back = c["op"] == "norm_backward"
        st["h"] = rows(M, H, 2.0)  # the residual stream (backward: after the block)
        st["y"] = rows(M, H, 0.5) if c["block"] else None
        st["post"] = (1.0 + 0.1 * _normal(g, H)).to(dt) if c["post"] else None
        st["gate"] = {"none": None, "channel": (0.5 + 0.1 * _normal(g, H)).to(dt),
                      "token": torch.sigmoid(_normal(g, M, 1)).to(dt)}[c["gate"]]
        st["scale"] = 0.7 if c["block"] else 1.0
        st["pre"] = (1.0 + 0.1 * _normal(g, H)).to(dt) if c["pre"] else None
        if back:
            st["dh_out"] = rows(M, H, 0.01)
            st["dx"] = rows(M, H, 0.01) if c["pre"] else None
        return st

    E, k = c["E"], c["topk"]
    P = M * k
    score, ids = torch.topk(_logits(g, c), k, dim=1)
    st["ids"] = ids.to(torch.int32)
    if "I" not in c:
        st["weights"] = torch.softmax(score, 1) if c["weighted"] else None
        st["al"] = _alignment(st["ids"], E, c["block_m"])
        cap = st["al"]["sorted_ids"].numel()
        st["pair_row"] = _pair_row(st["al"], P).view(M, k)
        if c["op"] == "permute":
            st["x"] = rows(M, H)
            st["pair_row_out"] = torch.empty(M, k, dtype=torch.int32, device="cuda")
        else:
            st["rows"] = rows(cap, H, 0.5)
        if c["op"] == "unpermute_backward":
            st["dout"] = rows(M, H, 0.01)
        # (rows behind the last expert's are not written: a program's buffer has what it had)
        st["rows_out"] = torch.zeros(cap, H, dtype=dt, device="cuda") if c["op"] != "unpermute" else None
        return st

    I = c["I"]
    st["al"] = _alignment(st["ids"], E, _tile_rows(c))
    if c["op"] == "gate_up" or c["op"] == "dx":
        up = c["op"] == "gate_up" or c["through"] == "gate_up"
        shape = (2 * I, H) if up else (H, I)
        st["w"] = torch.empty(E, *shape, dtype=dt, device="cuda")
        for e in range(E):
            st["w"][e] = rows(*shape, 0.02)
    if c["op"] == "gate_up" or (c["op"] == "dw" and c["through"] == "gate_up"):
        st["x"] = rows(M, H)
    if c["op"] in ("dx", "dw"):
        st["dc"] = rows(P, H if c["through"] == "down" else 2 * I, 0.01)
        if c["through"] == "down":
            z = _normal(g, P, 2 * I) * (0.02 * math.sqrt(H))
            st["z" if c["op"] == "dx" else "act"] = (z if c["op"] == "dx" else
                                                     z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]).to(dt)
    return st


def _pair_row(al, P):
    """The row of every pair in expert order."""
    s = al["sorted_ids"]
    at = torch.empty(P + 1, dtype=torch.int32, device=s.device)
    at[s.long()] = torch.arange(s.numel(), dtype=torch.int32, device=s.device)
    return at[:P]


# --------------------------------------------------------------------- run

def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


def _run_own(st):
    import moe_layer_topk_amd as moe
    c = st["case"]
    op = c["op"]
    if op == "permute":
        return moe.moe_permute(st["x"], st["ids"], st["al"], weights=st["weights"], rows=st["rows_out"],
                               pair_row=st["pair_row_out"])
    if op == "unpermute":
        return moe.moe_unpermute(st["rows"], st["pair_row"], weights=st["weights"])
    if op == "unpermute_backward":
        return moe.moe_unpermute_backward(st["dout"], st["rows"], st["weights"], st["pair_row"], st["al"],
                                          drows=st["rows_out"])
    if op == "norm":
        out = moe.moe_residual_norm(st["h"], st["y"], post_weight=st["post"], gate=st["gate"], scale=st["scale"],
                                    pre_weight=st["pre"], eps=EPS)
        return _given(out if c["block"] else (None, out[1]))
    if op == "norm_backward":
        return _given(moe.moe_residual_norm_backward(st["h"], st["dh_out"], st["dx"], st["y"], post_weight=st["post"],
                                                     gate=st["gate"], scale=st["scale"], pre_weight=st["pre"], eps=EPS))
    if op == "gate_up":
        return moe.moe_grouped_gemm(moe.MOE_GEMM_GATE_UP, st["x"], st["w"], st["al"], c["M"], c["topk"])[0]
    kind = moe.MOE_GEMM_DOWN if c["through"] == "down" else moe.MOE_GEMM_GATE_UP
    if op == "dx":
        return _given(moe.moe_grouped_gemm_dx(kind, st["dc"], st["w"], st["al"], c["M"], c["topk"], z=st.get("z")))
    return moe.moe_grouped_gemm_dw(kind, st["dc"], st["act" if c["through"] == "down" else "x"], st["al"], c["M"],
                                   c["topk"], dtype=TYPES[c["out"]])


def _given(outs):
    return [t for t in outs if t is not None]


def _plain_permute(st):
    c = st["case"]
    M, k, H = c["M"], c["topk"], c["H"]
    at = _pair_row(st["al"], M * k)
    v = st["x"].float()[:, None, :].expand(M, k, H)
    if st["weights"] is not None:
        v = v * st["weights"][:, :, None]
    rows = st["rows_out"].zero_()
    rows[at.long()] = v.reshape(M * k, H).to(rows.dtype)
    return rows, at.view(M, k)


def _plain_unpermute(st):
    v = st["rows"].float()[st["pair_row"].long()]
    if st["weights"] is not None:
        v = v * st["weights"][:, :, None]
    return v.sum(1).to(st["rows"].dtype)


def _plain_unpermute_backward(st):
    c = st["case"]
    at = st["pair_row"].long()
    d = st["dout"].float()[:, None, :]
    drows = st["rows_out"].zero_()
    drows[at.view(-1)] = (d * st["weights"][:, :, None]).reshape(-1, c["H"]).to(drows.dtype)
    return drows, (st["rows"].float()[at] * d).sum(2)


def _plain_norm(st):
    h = st["h"].float()
    outs = []
    if st["y"] is not None:
        u = st["y"].float()
        if st["post"] is not None:
            u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * st["post"].float()
        u = u * st["scale"]
        h = h + (u if st["gate"] is None else u * st["gate"].float())
        outs.append(h.to(st["h"].dtype))
    if st["pre"] is not None:
        outs.append((h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["pre"].float()).to(st["h"].dtype))
    return outs


def _norm_grad(d, v, w):
    """Gradients of v rsqrt(mean v^2 + eps) w for the gradient d: (of v, of w)."""
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    n, g = v * r, d * w
    return r * (g - n * (g * n).mean(1, keepdim=True)), (d * n).sum(0)


def _plain_norm_backward(st):
    dt = st["h"].dtype
    dh = st["dh_out"].float()
    dpost = dgate = dpre = dy = None
    if st["pre"] is not None:
        more, dpre = _norm_grad(st["dx"].float(), st["h"].float(), st["pre"].float())
        dh = dh + more
    if st["y"] is not None:
        y = st["y"].float()
        du = dh * st["scale"]
        u = y
        if st["post"] is not None:
            u = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * st["post"].float()
        if st["gate"] is not None:
            dgate = (du * u).sum(1, keepdim=True) if st["case"]["gate"] == "token" else (du * u).sum(0)
            du = du * st["gate"].float()
        dy = du
        if st["post"] is not None:
            dy, dpost = _norm_grad(du, y, st["post"].float())
        dy = dy.to(dt)
    return _given((dh.to(dt), dy, dpost, dgate, dpre))


def _by_expert(st, product):
    """Calls product(expert, its pairs) for every expert."""
    al = st["al"]
    first, count = al["expert_offsets"].tolist(), al["expert_counts"].tolist()
    for e, n in enumerate(count):
        product(e, al["sorted_ids"][first[e]:first[e] + n].long())


def _plain_gate_up(st):
    c = st["case"]
    x = st["x"].float()
    z = torch.empty(c["M"] * c["topk"], 2 * c["I"], dtype=st["x"].dtype, device=x.device)

    def product(e, p):
        if p.numel():
            z[p] = (x[p // c["topk"]] @ st["w"][e].float().t()).to(z.dtype)

    _by_expert(st, product)
    return z


def _plain_dx(st):
    c = st["case"]
    dc, I = st["dc"], c["I"]
    da = torch.empty(dc.shape[0], st["w"].shape[2], device=dc.device)

    def product(e, p):
        if p.numel():
            da[p] = dc[p].float() @ st["w"][e].float()

    _by_expert(st, product)
    if c["through"] == "gate_up":
        return [da.to(dc.dtype)]
    g, u = st["z"][:, :I].float(), st["z"][:, I:].float()
    s = 1.0 / (1.0 + torch.exp(-g))
    dz = torch.cat([da * u * s * (1.0 + g * (1.0 - s)), da * g * s], 1)
    return [dz.to(dc.dtype), (g * s * u).to(dc.dtype)]


def _plain_dw(st):
    c = st["case"]
    down = c["through"] == "down"
    a = st["act" if down else "x"]
    dw = torch.empty(c["E"], st["dc"].shape[1], a.shape[1], dtype=TYPES[c["out"]], device=a.device)

    def product(e, p):
        dw[e] = (st["dc"][p].float().t() @ a[p if down else p // c["topk"]].float()).to(dw.dtype)

    _by_expert(st, product)
    return dw


_PLAIN = {"permute": _plain_permute, "unpermute": _plain_unpermute, "unpermute_backward": _plain_unpermute_backward,
          "norm": _plain_norm, "norm_backward": _plain_norm_backward, "gate_up": _plain_gate_up, "dx": _plain_dx,
          "dw": _plain_dw}


# ------------------------------------------------------------------- exact
# The definitions in float64, written apart from the plain form above;
# gradients by torch's differentiation of the definition where memory allows.

def _exact_rows(st):
    """Pair by pair: the row of each is its place in the sorted list."""
    c = st["case"]
    s = st["al"]["sorted_ids"].long()
    r = (s < c["M"] * c["topk"]).nonzero().flatten()
    p = s[r]
    w = None if st["weights"] is None else st["weights"].double().reshape(-1)[p][:, None]
    return r, p, w


def _exact_norm(h, y, post, gate, scale, pre):
    def rms(v):
        return v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)

    out = h
    if y is not None:
        u = rms(y) * post if post is not None else y
        out = h + scale * (u * gate if gate is not None else u)
    return out, None if pre is None else rms(out) * pre


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    d = {k: v.double() for k, v in st.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if c["op"] in ("permute", "unpermute", "unpermute_backward"):
        r, p, w = _exact_rows(st)
        M, k, H = c["M"], c["topk"], c["H"]
        if c["op"] == "permute":
            rows = torch.zeros_like(d["rows_out"])
            rows[r] = d["x"][p // k] * (1.0 if w is None else w)
            at = torch.empty(M * k, dtype=torch.int32, device=r.device)
            at[p] = r.int()
            return rows, at.view(M, k)
        if c["op"] == "unpermute":
            out = d["rows"].new_zeros(M, H)
            return out.index_add_(0, p // k, d["rows"][r] * (1.0 if w is None else w))
        drows = torch.zeros_like(d["rows_out"])
        drows[r] = d["dout"][p // k] * w
        dw = d["rows"].new_empty(M * k)
        dw[p] = (d["dout"][p // k] * d["rows"][r]).sum(1)
        return drows, dw.view(M, k)
    if c["op"] == "norm":
        h, x = _exact_norm(d["h"], d.get("y"), d.get("post"), d.get("gate"), st["scale"], d.get("pre"))
        return _given((h if c["block"] else None, x))
    if c["op"] == "norm_backward":
        # the stream before the block, so that the one after it is the given one
        y, post, gate, pre = (t.requires_grad_() if t is not None else None
                              for t in (d.get("y"), d.get("post"), d.get("gate"), d.get("pre")))
        with torch.no_grad():
            step = _exact_norm(torch.zeros_like(d["h"]), y, post, gate, st["scale"], None)[0]
        h = (d["h"] - step).requires_grad_()
        out, x = _exact_norm(h, y, post, gate, st["scale"], pre)
        leaves = _given((h, y, post, gate, pre))
        outs, grads = ([out], [d["dh_out"]]) if x is None else ([out, x], [d["dh_out"], d["dx"]])
        return list(torch.autograd.grad(outs, leaves, grads))
    k, I = c["topk"], c["I"]
    owner = torch.empty(c["M"] * k, dtype=torch.long, device="cuda")
    owner[:] = st["ids"].reshape(-1)
    pairs = [(owner == e).nonzero().flatten() for e in range(c["E"])]
    if c["op"] == "gate_up":
        z = torch.empty(c["M"] * k, 2 * I, dtype=torch.float64, device="cuda")
        for e, p in enumerate(pairs):
            z[p] = torch.matmul(st["w"][e].double(), d["x"][p // k].t()).t()
        return z
    if c["op"] == "dx":
        da = torch.empty(c["M"] * k, st["w"].shape[2], dtype=torch.float64, device="cuda")
        for e, p in enumerate(pairs):
            da[p] = torch.matmul(st["w"][e].double().t(), d["dc"][p].t()).t()
        if c["through"] == "gate_up":
            return [da]
        z = d["z"].requires_grad_()
        act = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        return [torch.autograd.grad(act, z, da)[0], act.detach()]
    a = st["act" if c["through"] == "down" else "x"]
    dw = torch.empty(c["E"], st["dc"].shape[1], a.shape[1], dtype=torch.float64, device="cuda")
    for e, p in enumerate(pairs):
        rows = a[p if c["through"] == "down" else p // k].double()
        dw[e] = torch.matmul(rows.t(), d["dc"][p]).t()
    return dw
