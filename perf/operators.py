"""Cases of the operators around the layer's training and serving step: the choice
of experts from router logits and its gradient, the sequence-wise balance loss, 8-bit
activation checkpoints and the combine's gradient from them, and the gradient of
the router projection.

``own = False`` computes each case in plain torch operations, ``own = True``
through this package's entry points."""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # serving: one decode step of 32 sequences, group-limited sigmoid routing with a balancing bias
        {"name": "select decode", "op": "select", "T": 32, "E": 256, "k": 8, "score": "sigmoid", "groups": 8,
         "topk_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "bias": True, "dtype": "f32"},
        # the same rule on the prefill layer's 16384 tokens
        {"name": "select prefill", "op": "select", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "groups": 8,
         "topk_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "bias": True, "dtype": "f32"},
        # training: the prefill batch's combine-weight gradients and balance loss back to the logits, in one pass
        {"name": "select grad sigmoid", "op": "select_grad", "T": 16384, "E": 256, "k": 8, "score": "sigmoid",
         "renorm": True, "scale": 2.5, "dtype": "f32", "seqs": 4},
        # training a small softmax router whose weights are not renormalised (every logit gets a gradient)
        {"name": "select grad softmax", "op": "select_grad", "T": 2999, "E": 60, "k": 4, "score": "softmax",
         "renorm": False, "scale": 1.0, "dtype": "bf16", "seqs": 0},
        # balance loss and its gradient over a packed batch of ragged sequences
        {"name": "balance packed", "op": "balance", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "dtype": "f32",
         "seqs": 9},
        # a short batch of a smaller softmax router, one sequence
        {"name": "balance short", "op": "balance", "T": 1021, "E": 64, "k": 6, "score": "softmax", "dtype": "bf16",
         "seqs": 1},
        # the prefill layer's routed outputs (T*k rows) kept in e4m3 tiles and read back
        {"name": "checkpoint routed outputs", "op": "checkpoint", "rows": 131072, "cols": 7168, "format": "e4m3",
         "dtype": "bf16"},
        # a small fp32 activation of odd width in 8-bit integers
        {"name": "checkpoint odd", "op": "checkpoint", "rows": 301, "cols": 1001, "format": "i8", "dtype": "f32"},
        # the combine's gradient of the prefill layer from e4m3 checkpoints
        {"name": "combine grad prefill", "op": "combine_grad", "T": 16384, "d": 7168, "format": "e4m3"},
        # the mid-size layer's, from 8-bit integers
        {"name": "combine grad mid", "op": "combine_grad", "T": 2048, "d": 2048, "format": "i8"},
        # the router projection's gradient of the prefill layer
        {"name": "router grad prefill", "op": "router_grad", "T": 16384, "d": 7168, "dtype": "bf16"},
        # a small ragged batch of a narrow layer
        {"name": "router grad small", "op": "router_grad", "T": 301, "d": 896, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select_grad", "balance", "checkpoint", "combine_grad", "router_grad"])
    if op == "checkpoint":
        return {"op": op, "rows": _log(rng, 1, 65536), "cols": _log(rng, 1, 8192), "format": rng.choice(["e4m3", "i8"]),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "combine_grad":
        return {"op": op, "T": _log(rng, 1, 16384), "d": 64 * _log(rng, 1, 64), "format": rng.choice(["e4m3", "i8", "bf16"])}
    if op == "router_grad":
        return {"op": op, "T": _log(rng, 1, 16384), "d": 128 * _log(rng, 1, 32), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    groups = rng.choice([1, 1, 2, 4, 8]) if op == "select" else 1
    per = rng.randint(max(2, 8 // groups), 512 // groups)
    E = groups * per
    topk_groups = rng.randint((groups + 1) // 2, groups)
    k = rng.randint(1, min(16, topk_groups * per))
    c = {"op": op, "T": _log(rng, 1, 32768 if E <= 256 else 16384), "E": E, "k": k, "score": rng.choice(["sigmoid", "softmax"]),
         "dtype": rng.choice(["f32", "bf16"])}
    if op == "select":
        c.update(groups=groups, topk_groups=topk_groups, group_score=rng.choice(["max", "top2"]),
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), bias=rng.random() < 0.6)
    elif op == "select_grad":
        c.update(renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), seqs=rng.choice([0, 1, rng.randint(2, 64)]))
    else:
        c["seqs"] = rng.choice([1, rng.randint(2, 64)])
    return c


# ---------------------------------------------------------------- the inputs

TILE = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ALPHA = 1e-2


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1000003 * seed + 7)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _logits(c, g):
    """Router logits: unit-scale products with a preference per expert."""
    return (1.2 * _normal(g, c["T"], c["E"]) + 0.6 * _normal(g, c["E"])).to(TYPES[c["dtype"]])


def _some_ids(c, g):
    """k distinct experts for each token, ascending."""
    return torch.rand(c["T"], c["E"], generator=g, device=DEV).topk(c["k"], dim=1).indices.sort(dim=1).values.to(torch.int32)


def _sequences(c, g):
    """Offsets of c["seqs"] ragged sequences packed into the batch (some may be empty)."""
    cuts = torch.randint(0, c["T"] + 1, (c["seqs"] - 1,), generator=g, device=DEV).sort().values
    ends = torch.tensor([0, c["T"]], device=DEV)
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _of_sequence(off, T):
    """The sequence that each token lies in."""
    return torch.searchsorted(off[1:].contiguous(), torch.arange(T, device=DEV, dtype=torch.int32), right=True)


def _tiles(x, fmt):
    """x [rows, cols] in 8-bit tiles of 128 columns: codes and the tiles' exponents (E8M0 bytes)."""
    rows, cols = x.shape
    n = -(-cols // TILE)
    v = torch.nn.functional.pad(x.float(), (0, n * TILE - cols)).view(rows, n, TILE)
    top = 448.0 if fmt == "e4m3" else 127.0
    amax = v.abs().amax(dim=2)
    m, e = torch.frexp(amax.double() / top)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-126, 127)
    q = torch.ldexp(v, -e[..., None])
    q = q.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "e4m3" else torch.round(q).to(torch.int8).view(torch.uint8)
    return q.view(rows, n * TILE)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _values(codes, scales, fmt):
    """What 8-bit tiles stand for, in fp32."""
    v = codes.view(torch.float8_e4m3fn).float() if fmt == "e4m3" else codes.view(torch.int8).float()
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return v * s.repeat_interleave(TILE, dim=1)[:, : codes.shape[1]]


def _f32(*shape):
    return torch.empty(*shape, dtype=torch.float32, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    op = c["op"]
    if op in ("select", "select_grad", "balance"):
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = _logits(c, g)
        if op == "select":
            s["bias"] = 0.1 * torch.rand(E, generator=g, device=DEV) - 0.05 if c["bias"] else None
            s["idx"], s["weights"] = torch.empty(T, k, dtype=torch.int32, device=DEV), _f32(T, k)
            return s
        s["idx"], s["dlogits"] = _some_ids(c, g), _f32(T, E)
        if op == "select_grad":
            s["dweights"] = _normal(g, T, k)
        if c["seqs"]:
            s["seq"] = _sequences(c, g)
            s["dloss"] = 0.5 + torch.rand(c["seqs"], generator=g, device=DEV)
            s["loss"], s["load"] = _f32(c["seqs"]), _f32(c["seqs"], E)
            if op == "select_grad":  # the loads that the forward's loss left
                s["load"].copy_(2.0 * torch.rand(c["seqs"], E, generator=g, device=DEV))
    elif op == "checkpoint":
        x = _normal(g, c["rows"], c["cols"]).mul_(torch.exp(_normal(g, c["rows"], 1)))
        s["x"] = x.to(TYPES[c["dtype"]])
        s["codes"] = torch.empty(c["rows"], c["cols"], dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(c["rows"], -(-c["cols"] // TILE), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty_like(s["x"])
    elif op == "combine_grad":
        T, d, k = c["T"], c["d"], 8
        y = _normal(g, T * k, d)
        s["y"], s["scales"] = (y.bfloat16(), None) if c["format"] == "bf16" else _tiles(y, c["format"])
        del y
        s["dy"] = _normal(g, T, d)
        ids = _some_ids({"T": T, "E": 256, "k": k}, g)
        s["row_of"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        order = ids.reshape(-1).sort(stable=True).indices
        s["row_of"][order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.1
        s["weights"] = w / w.sum(dim=1, keepdim=True)
        s["dy_perm"], s["dg"] = torch.empty(T * k, d, dtype=torch.bfloat16, device=DEV), _f32(T, k)
    else:
        T, d = c["T"], c["d"]
        s["x"] = _normal(g, T, d).to(TYPES[c["dtype"]])
        s["w"] = _normal(g, 256, d) * d ** -0.5
        s["dlogits"] = 1e-2 * _normal(g, T, 256)
        s["dx_in"] = 0.1 * _normal(g, T, d)
        s["dx"], s["dw"] = _f32(T, d), _f32(256, d)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](c, state)


def _scores(x, kind):
    return torch.sigmoid(x) if kind == "sigmoid" else torch.softmax(x, dim=1)


def _plain_select(c, s):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    far = s["logits"].double()  # the choice in 64 bits: scores next to the border decide whole numbers
    wide = _scores(far, c["score"])
    key = wide + s["bias"].double() if c["bias"] else far  # without a bias the scores' order is the logits'
    if c["topk_groups"] < G:
        by = key if c["bias"] or c["group_score"] == "max" else wide
        by = by.view(T, G, E // G).topk(1 if c["group_score"] == "max" else min(2, E // G), dim=2).values.sum(dim=2)
        best = by.sort(dim=1, descending=True, stable=True).indices[:, : c["topk_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        key = key.masked_fill(~open_.repeat_interleave(E // G, dim=1), -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :k].sort(dim=1).values
    w = _scores(s["logits"].float(), c["score"]).gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"idx": idx.to(torch.int32), "weights": w * c["scale"]}


def _dscores_to_dlogits(p, dp, kind):
    if kind == "sigmoid":
        return dp * p * (1 - p)
    return p * (dp - (dp * p).sum(dim=1, keepdim=True))


def _weights_grad(c, s, p):
    """The combine weights' gradient with respect to the scores, [T, E]."""
    at = s["idx"].long()
    dw = s["dweights"] * c["scale"]
    if c["renorm"]:
        chosen = p.gather(1, at)
        total = chosen.sum(dim=1, keepdim=True)
        dw = (dw - (dw * chosen).sum(dim=1, keepdim=True) / total) / total
    return torch.zeros_like(p).scatter_(1, at, dw)


def _balance_grad(c, s, p, load):
    """The balance loss's gradient with respect to the scores, [T, E]."""
    at = _of_sequence(s["seq"], c["T"])
    n = (s["seq"][1:] - s["seq"][:-1]).clamp(min=1).float()
    dn = (load * (ALPHA * s["dloss"] / n)[:, None])[at]
    total = p.sum(dim=1, keepdim=True)
    return (dn - (dn * p).sum(dim=1, keepdim=True) / total) / total


def _plain_select_grad(c, s):
    p = _scores(s["logits"].float(), c["score"])
    dp = _weights_grad(c, s, p)
    if c["seqs"]:
        dp = dp + _balance_grad(c, s, p, s["load"])
    return {"dlogits": _dscores_to_dlogits(p, dp, c["score"])}


def _sequence_sums(x, off):
    """Each sequence's sums of the rows of x, as a product with the sequences' membership."""
    inside = _of_sequence(off, x.shape[0]) == torch.arange(off.numel() - 1, device=DEV)[:, None]
    return (inside.float() @ x).double()


def _plain_balance(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    p = _scores(s["logits"].float(), c["score"])
    n = (s["seq"][1:] - s["seq"][:-1]).clamp(min=1)
    load = _sequence_sums(torch.zeros_like(p).scatter_(1, s["idx"].long(), 1.0), s["seq"]) * (E / (k * n.double()))[:, None]
    share = _sequence_sums(p / p.sum(dim=1, keepdim=True), s["seq"])
    loss = ALPHA * (load * share).sum(dim=1) / n
    load = load.float()
    return {"loss": loss.float(), "load": load, "dlogits": _dscores_to_dlogits(p, _balance_grad(c, s, p, load), c["score"])}


def _plain_checkpoint(c, s):
    codes, scales = _tiles(s["x"], c["format"])
    return {"scales": scales, "values": _values(codes, scales, c["format"]).to(s["x"].dtype)}


def _plain_combine_grad(c, s):
    T, d = c["T"], c["d"]
    y = s["y"].float() if c["format"] == "bf16" else _values(s["y"], s["scales"], c["format"])
    at = s["row_of"].long()
    dg = torch.bmm(y[at].view(T, 8, d), s["dy"].view(T, d, 1)).view(T, 8)
    out = torch.empty(T * 8, d, dtype=torch.bfloat16, device=DEV)
    out[at] = (s["weights"][:, :, None] * s["dy"][:, None, :]).view(T * 8, d).bfloat16()
    return {"dy_perm": out, "dg": dg}


def _plain_router_grad(c, s):
    return {"dx": torch.addmm(s["dx_in"], s["dlogits"], s["w"]), "dw": s["dlogits"].t() @ s["x"].float()}


_PLAIN = {"select": _plain_select, "select_grad": _plain_select_grad, "balance": _plain_balance,
          "checkpoint": _plain_checkpoint, "combine_grad": _plain_combine_grad, "router_grad": _plain_router_grad}


def _selection(moe, c):
    return moe.selection(c["T"], c["E"], c["k"], score=c["score"], n_group=c.get("groups", 1),
                         topk_group=c.get("topk_groups", 1), group_score=c.get("group_score", "max"),
                         renorm=c.get("renorm", True), scale=c.get("scale", 1.0), logits=c["dtype"])


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _own_select(c, s):
    import sparse_expert_routing_amd as moe
    moe.moe_select(_selection(moe, c), s["logits"], s["bias"], s["idx"], s["weights"])
    return {"idx": s["idx"], "weights": s["weights"]}


def _own_select_grad(c, s):
    import sparse_expert_routing_amd as moe
    moe.moe_select_backward(_selection(moe, c), s["logits"], s["idx"], s["dweights"], s["dlogits"], seq_offsets=s.get("seq"),
                            load=s.get("load"), dloss=s.get("dloss"), alpha=ALPHA)
    return {"dlogits": s["dlogits"]}


def _own_balance(c, s):
    import sparse_expert_routing_amd as moe
    sel = _selection(moe, c)
    ws = _bytes(moe.balance_workspace_bytes(sel, c["seqs"]))
    moe.moe_balance_loss(sel, s["logits"], s["idx"], s["seq"], ALPHA, s["loss"], s["load"], ws)
    moe.moe_select_backward(sel, s["logits"], s["idx"], None, s["dlogits"], seq_offsets=s["seq"], load=s["load"],
                            dloss=s["dloss"], alpha=ALPHA)
    return {"loss": s["loss"], "load": s["load"], "dlogits": s["dlogits"]}


def _own_checkpoint(c, s):
    import sparse_expert_routing_amd as moe
    moe.moe_checkpoint_pack(s["x"], s["codes"], s["scales"], c["format"])
    moe.moe_checkpoint_unpack(s["codes"], s["scales"], c["format"], s["out"])
    return {"scales": s["scales"], "values": s["out"]}


def _own_combine_grad(c, s):
    import sparse_expert_routing_amd as moe
    ds = moe.desc(c["T"], c["d"], 256, 8, 128)
    moe.moe_combine_backward(ds, s["dy"], moe.saved(s["y"], s["scales"], c["format"]), s["row_of"], s["weights"], s["dy_perm"],
                             s["dg"])
    return {"dy_perm": s["dy_perm"], "dg": s["dg"]}


def _own_router_grad(c, s):
    import sparse_expert_routing_amd as moe
    ds = moe.desc(c["T"], c["d"], 256, 8, 128, c["dtype"], c["dtype"])
    ws = _bytes(moe.workspace_bytes(ds, moe.MOE_WS_ROUTER_GRAD))
    moe.moe_router_logits_backward(ds, s["x"], s["w"], s["dlogits"], s["dx_in"], s["dx"], s["dw"], ws)
    return {"dx": s["dx"], "dw": s["dw"]}


_OWN = {"select": _own_select, "select_grad": _own_select_grad, "balance": _own_balance, "checkpoint": _own_checkpoint,
        "combine_grad": _own_combine_grad, "router_grad": _own_router_grad}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    size = 2 if c.get("dtype") == "bf16" else 4
    if op in ("select", "select_grad", "balance"):
        T, E, k = c["T"], c["E"], c["k"]
        if op == "select":
            return {"bytes": T * E * size + 8 * T * k + 4 * E * c["bias"], "flops": 6 * T * E}
        dense = op == "balance" or c["seqs"] or (c["score"] == "softmax" and not c["renorm"])
        read = T * E * size if dense else T * k * size
        return {"bytes": read + 4 * T * E + (8 if op == "select_grad" else 4) * T * k + 4 * c["seqs"] * (E + 3), "flops": 10 * T * E}
    if op == "checkpoint":
        n, tiles = c["rows"] * c["cols"], c["rows"] * -(-c["cols"] // TILE)
        return {"bytes": 2 * n * size + 2 * (n + tiles), "flops": 6 * n}
    if op == "combine_grad":
        n = c["T"] * c["d"]
        return {"bytes": 4 * n + 8 * n * (2 if c["format"] == "bf16" else 1 + 1 / 128) + 16 * n + 8 * 12 * c["T"], "flops": 24 * n}
    n = c["T"] * c["d"]
    return {"bytes": n * (size + 8) + 4 * 256 * (c["T"] + 2 * c["d"]), "flops": 4 * 256 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "select":
        return _exact_select(c, s)
    if op == "select_grad":
        return {"dlogits": _exact_dlogits(c, s, s["dweights"].double(), s["load"].double() if c["seqs"] else None)}
    if op == "balance":
        return _exact_balance(c, s)
    if op == "checkpoint":
        return {"scales": None, "values": _exact_values(s["x"].double(), c["format"])}
    if op == "combine_grad":
        return _exact_combine_grad(c, s)
    dl = s["dlogits"].double()
    return {"dx": s["dx_in"].double() + dl @ s["w"].double(), "dw": dl.t() @ s["x"].double()}


def _probabilities(l, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _exact_select(c, s):
    """By rank counting: an expert's rank is the number of those ahead of it."""
    T, E, G, per = c["T"], c["E"], c["groups"], c["E"] // c["groups"]
    out = []
    for l in s["logits"].double().split(max(1, (1 << 26) // (E * E))):
        p = _probabilities(l, c["score"])
        a = p + s["bias"].double() if c["bias"] else p
        g = torch.zeros(l.shape[0], G, dtype=torch.float64, device=DEV)
        for i in range(G):
            part = a[:, i * per : (i + 1) * per].sort(dim=1).values
            g[:, i] = part[:, -1] + (part[:, -2] if c["group_score"] == "top2" and per > 1 else 0)
        is_open = (_ranks(g) < c["topk_groups"])[:, torch.arange(E, device=DEV) // per]
        a = torch.where(is_open, a, torch.full_like(a, -1e300))
        take = _ranks(a) < c["k"]
        w = p[take].view(-1, c["k"])
        out.append(w / w.sum(dim=1, keepdim=True) if c["renorm"] else w)
    return {"idx": None, "weights": torch.cat(out) * c["scale"]}


def _ranks(a):
    n = torch.arange(a.shape[1], device=DEV)
    ahead = (a[:, None, :] > a[:, :, None]) | ((a[:, None, :] == a[:, :, None]) & (n[None, :] < n[:, None]))
    return ahead.sum(dim=2)


def _exact_dlogits(c, s, dw, load):
    """Gradients through the Jacobians, written for the logits directly."""
    l = s["logits"].double()
    T, E = l.shape
    z = _probabilities(l, c["score"])
    out = torch.zeros_like(l)
    if dw is not None:
        at = s["idx"].long()
        if c["score"] == "softmax" and not c["renorm"]:  # w_j = scale p_j
            g = torch.zeros_like(l).scatter_(1, at, dw * c["scale"])
            out += z * g - z * (z * g).sum(dim=1, keepdim=True)
        else:
            zc = z.gather(1, at)
            slope = 1 - zc if c["score"] == "sigmoid" else torch.ones_like(zc)  # d log(score) / d logit, up to a common term
            if c["renorm"]:  # w_j = scale r_j, with r the shares among the chosen
                r = zc / zc.sum(dim=1, keepdim=True)
                g = c["scale"] * r * (dw - (dw * r).sum(dim=1, keepdim=True)) * slope
            else:
                g = c["scale"] * dw * zc * slope
            out.scatter_add_(1, at, g)
    if load is not None:
        off = s["seq"].tolist()
        share = z / z.sum(dim=1, keepdim=True)
        for q in range(len(off) - 1):
            a, b = off[q], off[q + 1]
            if a == b:
                continue
            f = ALPHA * s["dloss"][q].double() * load[q] / (b - a)
            r = share[a:b]
            g = r * (f - (r * f).sum(dim=1, keepdim=True))
            out[a:b] += g * (1 - z[a:b]) if c["score"] == "sigmoid" else g
    return out


def _exact_balance(c, s):
    off, E = s["seq"].tolist(), c["E"]
    p = _probabilities(s["logits"].double(), c["score"])
    p = p / p.sum(dim=1, keepdim=True)
    loss, load = [], []
    for a, b in zip(off, off[1:]):
        f = torch.bincount(s["idx"][a:b].reshape(-1).long(), minlength=E).double() * E / (c["k"] * max(1, b - a))
        load.append(f)
        loss.append(ALPHA * (f * p[a:b].sum(dim=0)).sum() / max(1, b - a))
    load = torch.stack(load)
    return {"loss": torch.stack(loss), "load": load, "dlogits": _exact_dlogits(c, s, None, load)}


def _exact_values(x, fmt):
    """Each value rounded to its tile's grid: steps of 2^-3 of its binade (e4m3) or of the scale (integers)."""
    out = torch.empty_like(x)
    top = 448.0 if fmt == "e4m3" else 127.0
    for lo in range(0, x.shape[1], TILE):
        v = x[:, lo : lo + TILE]
        a = v.abs().amax(dim=1, keepdim=True)
        scale = torch.where(a > 0, torch.exp2(torch.ceil(torch.log2(a / top) - 1e-13)), torch.ones_like(a))
        u = v / scale
        if fmt == "e4m3":
            step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0**-6))) - 3)
            out[:, lo : lo + TILE] = torch.round(u / step) * step * scale
        else:
            out[:, lo : lo + TILE] = torch.round(u) * scale
    return out


def _exact_combine_grad(c, s):
    T, d = c["T"], c["d"]
    dg = torch.empty(T * 8, dtype=torch.float64, device=DEV)
    out = torch.empty(T * 8, d, dtype=torch.float64, device=DEV)
    token = torch.arange(T, device=DEV)
    for j in range(8):
        for part in token.split(4096):
            row = s["row_of"].view(T, 8)[part, j].long()
            y = s["y"][row]
            if c["format"] == "bf16":
                y = y.double()
            else:
                v = y.view(torch.float8_e4m3fn if c["format"] == "e4m3" else torch.int8).double()
                y = v * torch.exp2(s["scales"][row].double() - 127).repeat_interleave(TILE, dim=1)[:, :d]
            dy = s["dy"][part].double()
            dg[part * 8 + j] = (y * dy).sum(dim=1)
            out[row] = dy * s["weights"][part, j, None].double()
    return {"dy_perm": out, "dg": dg.view(T, 8)}
