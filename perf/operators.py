"""Cases of the operators that train a sparse block: what each computes in plain torch
operations, and the same through the framework's training entry points.

The operators are the dispatch (token rows sorted by expert and back, with the router weights,
and both gradients), the experts' grouped products with their gradients, the norms before and
after the block fused with its gate and residual scale, and the router's gradient. `listed()`
gives the fixed cases, `draw()` more of the same ranges; sizes follow the workloads of
`moe_inputs` (Mixtral-, gpt-oss-, Qwen3- and DeepSeek-V3-shaped layers) or are generic.
"""
import math

import torch

own = False

DEV = "cuda"
PAD = 16  # an expert's run of rows is padded to a multiple of this
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 8 requests: the experts' rows go back to their tokens; latency
        dict(name="unpermute-decode", op="unpermute", T=8, k=4, E=128, H=2880, dtype="bf16", skew=1.0,
             dropped=0.0),
        # a prefill batch or training micro-batch with many small experts: sort and copy
        dict(name="permute-many-experts", op="permute", T=4096, k=8, E=256, H=7168, dtype="bf16", skew=0.5,
             dropped=0.0),
        # gradient of the copy in fp32, an odd batch in which some slots were dropped
        dict(name="permute-backward-f32-odd", op="permute_backward", T=1531, k=3, E=37, H=2056, dtype="f32",
             skew=1.0, dropped=0.1),
        # gradient of the weighted sum of a long training batch with skewed loads
        dict(name="unpermute-backward-skewed", op="unpermute_backward", T=8192, k=8, E=128, H=4096,
             dtype="bf16", skew=1.5, dropped=0.0),
        # forward and backward of the experts where every expert sees a handful of rows: the
        # weights' bytes bound it
        dict(name="experts-few-rows", op="experts", T=24, k=4, E=32, H=2880, I=2880, dtype="bf16", skew=0.3),
        # forward and backward of eight large experts on a full batch: the products bound it
        dict(name="experts-large", op="experts", T=4096, k=2, E=8, H=4096, I=14336, dtype="bf16", skew=0.1),
        # fp32 weight gradient (as a master gradient is kept) over ragged runs of rows
        dict(name="weight-grad-f32-ragged", op="weight_grad", T=8191, k=8, E=128, M=4096, N=1536, dtype="bf16",
             skew=0.5),
        # one token's residual join and the next block's norm: latency
        dict(name="join-one-token", op="join", T=1, H=4096, dtype="bf16", gate="channel", scale=0.5, offset=0.0),
        # the join of a training batch with a full gate
        dict(name="join-batch-gated", op="join", T=8192, H=7168, dtype="bf16", gate="full", scale=1.0, offset=0.0),
        # its gradient, with a gate a token and a norm weight stored as an offset from one
        dict(name="join-backward-batch", op="join_backward", T=8192, H=4096, dtype="bf16", gate="token", scale=0.7,
             offset=1.0),
        # gradient of grouped-sigmoid routing over a batch
        dict(name="route-backward-sigmoid", op="route_backward", T=4096, E=256, k=8, mode=1, renormalize=True,
             scale=2.5),
        # gradient of a softmax over all experts (weights not renormalised), few tokens
        dict(name="route-backward-softmax", op="route_backward", T=61, E=128, k=4, mode=0, renormalize=False,
             scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["permute", "permute_backward", "unpermute", "unpermute_backward", "experts", "experts",
                     "weight_grad", "norm", "norm_backward", "join", "join_backward", "route_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    E = _log(rng, 2, 256)
    k = rng.randint(1, min(E, 8))
    if op in ("permute", "permute_backward", "unpermute", "unpermute_backward"):
        return dict(op=op, T=_log(rng, 1, 6000), k=k, E=E, H=8 * _log(rng, 8, 896), dtype=dtype,
                    skew=round(rng.uniform(0, 1.5), 2), dropped=rng.choice([0.0, 0.0, 0.15]))
    if op == "experts":
        T, H, I = _log(rng, 1, 4096), 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1024)
        E = min(E, max(2, 400_000_000 // (H * I)))
        k = min(k, E)
        most = 2 * 4096 * 4096 * 14336 // (16 if dtype == "f32" else 2)
        T = max(1, min(T, most // (k * H * I)))
        return dict(op=op, T=T, k=k, E=E, H=H, I=I, dtype=dtype, skew=round(rng.uniform(0, 0.5), 2))
    if op == "weight_grad":
        M, N = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 512)
        E = min(E, max(2, 800_000_000 // (M * N)))
        k = min(k, E)
        return dict(op=op, T=_log(rng, 1, 8192), k=k, E=E, M=M, N=N, dtype=dtype,
                    skew=round(rng.uniform(0, 0.5), 2))
    if op == "route_backward":
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, mode=rng.randint(0, 1),
                    renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    c = dict(op=op, T=_log(rng, 1, 8192), H=8 * _log(rng, 8, 896), dtype=dtype, offset=rng.choice([0.0, 1.0]))
    if op.startswith("join"):
        c |= dict(gate=rng.choice(["none", "channel", "token", "full"]), scale=rng.choice([1.0, 0.5]))
    return c


# ----------------------------------------------------------------------------------- inputs
def max_rows(c):
    n = c["T"] * c["k"]
    return (n + min(c["E"], n) * (PAD - 1)) // PAD * PAD


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _ids(c, g):
    """Distinct experts a token from skewed scores, the best first, some slots dropped (-1)."""
    T, k, E = c["T"], c["k"], c["E"]
    u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
    score = torch.randn(E, generator=g, device=DEV) * c["skew"] - torch.log(-torch.log(u))
    ids = score.topk(k, dim=1).indices.to(torch.int32)
    if c.get("dropped"):
        ids[torch.rand(T, k, generator=g, device=DEV) < c["dropped"]] = -1
    return ids


def sort_table(ids, E, P):
    """Where every routed slot goes: rows of one expert together, slots in order, runs padded."""
    n = ids.numel()
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    padded = (counts + PAD - 1) // PAD * PAD
    base = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(counts, 0) - counts
    ks = key[order]
    row = base[ks] + torch.arange(n, device=ids.device) - first[ks]
    row = torch.where(ks < E, row, P)
    sorted_ids = torch.full((P + 1,), n, dtype=torch.int32, device=ids.device)
    sorted_ids[row] = order.to(torch.int32)
    pos = torch.empty(n, dtype=torch.long, device=ids.device)
    pos[order] = torch.where(ks < E, row, -1)
    return sorted_ids[:P].contiguous(), pos.to(torch.int32).view(ids.shape), counts[:E].to(torch.int32)


def _weights(c, g):
    return torch.softmax(_randn(g, c["T"], c["k"]), 1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, s = c["op"], {"case": c}
    dt = TYPES[c.get("dtype", "f32")]
    if op == "route_backward":
        s["logits"] = _randn(g, c["T"], c["E"], std=1.5)
        s["logit_bias"] = _randn(g, c["E"], std=0.5) if c["mode"] == 0 else None
        key = s["logits"] + s["logit_bias"] if c["mode"] == 0 else torch.sigmoid(s["logits"])
        s["topk_ids"] = key.topk(c["k"], dim=1).indices.to(torch.int32)
        s["dtopk_w"] = _randn(g, c["T"], c["k"])
        return s
    if op in ("norm", "norm_backward", "join", "join_backward"):
        T, H = c["T"], c["H"]
        one = 1.0 - c["offset"]
        s["x"] = _randn(g, T, H, dtype=dt, std=2.0)
        s["gamma"] = one + _randn(g, H, std=0.2)
        if op == "norm_backward":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dh"] = _randn(g, T, H, dtype=dt)
            s["dres"] = _randn(g, T, H, dtype=dt)
        if op.startswith("join"):
            s["y"] = _randn(g, T, H, dtype=dt)
            s["gamma_next"] = one + _randn(g, H, std=0.2)
            shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[c["gate"]]
            s["gate"] = None if shape is None else torch.sigmoid(_randn(g, *shape)).to(
                dt if c["gate"] == "full" else torch.float32)
        if op == "join_backward":  # what the forward pass left, and the gradients that come in
            s["out"], s["rstd_y"], _, s["rstd_out"] = _join(s, torch.float32)
            s["dres"] = _randn(g, T, H, dtype=dt)
            s["dh"] = _randn(g, T, H, dtype=dt)
        return s
    P = max_rows(c)
    ids = _ids(c, g)
    s["sorted_ids"], s["row_pos"], s["counts"] = sort_table(ids, c["E"], P)
    if op == "permute":
        s["topk_ids"] = ids
        s["x"] = _randn(g, c["T"], c["H"], dtype=dt)
        return s
    live = (s["sorted_ids"] < c["T"] * c["k"]).unsqueeze(1)
    if op in ("experts", "weight_grad"):
        s["capacity"] = int(s["counts"].max())
    if op == "weight_grad":
        s["dy"] = _randn(g, P, c["M"], dtype=dt) * live
        s["a"] = _randn(g, P, c["N"], dtype=dt) * live
    elif op == "experts":
        E, H, I = c["E"], c["H"], c["I"]
        s["xs"] = _randn(g, P, H, dtype=dt) * live
        s["dys"] = _randn(g, P, H, dtype=dt) * live
        s["W13"], s["W2"] = torch.empty(E, 2 * I, H, dtype=dt, device=DEV), torch.empty(E, H, I, dtype=dt, device=DEV)
        for e in range(E):
            s["W13"][e] = _randn(g, 2 * I, H, dtype=dt, std=H ** -0.5)
            s["W2"][e] = _randn(g, H, I, dtype=dt, std=I ** -0.5)
    elif op == "permute_backward":
        s["dxs"] = _randn(g, P, c["H"], dtype=dt) * live
    else:
        s["ys"] = _randn(g, P, c["H"], dtype=dt) * live
        s["topk_w"] = _weights(c, g)
        if op == "unpermute_backward":
            s["dout"] = _randn(g, c["T"], c["H"], dtype=dt)
    return s


# ------------------------------------------------------------------------------- plain forms
def _rows_of(v, row_pos):
    """v[row_pos] with zeros for dropped slots: [T, k, H] in 32 bits."""
    got = v[row_pos.clamp(min=0).long()].float()
    return got * (row_pos >= 0).unsqueeze(-1)


def _permute(s):
    c = s["case"]
    P, n = max_rows(c), c["T"] * c["k"]
    sorted_ids, pos, counts = sort_table(s["topk_ids"], c["E"], P)
    live = (sorted_ids < n).unsqueeze(1)
    xs = torch.where(live, s["x"][(sorted_ids.long() // c["k"]).clamp(max=c["T"] - 1)], 0)
    return {"xs": xs, "row_pos": pos, "sorted_ids": sorted_ids, "counts": counts}


def _permute_backward(s):
    return {"dx": _rows_of(s["dxs"], s["row_pos"]).sum(1).to(s["dxs"].dtype)}


def _unpermute(s):
    return {"out": (_rows_of(s["ys"], s["row_pos"]) * s["topk_w"].unsqueeze(-1)).sum(1).to(s["ys"].dtype)}


def _unpermute_backward(s):
    c = s["case"]
    n = c["T"] * c["k"]
    sid = s["sorted_ids"].long()
    at = sid.clamp(max=n - 1)
    w = torch.where(sid < n, s["topk_w"].reshape(-1)[at], 0.0)
    dys = (w.unsqueeze(1) * s["dout"][at // c["k"]].float()).to(s["ys"].dtype)
    dw = (_rows_of(s["ys"], s["row_pos"]) * s["dout"].float().unsqueeze(1)).sum(-1)
    return {"dys": dys, "dtopk_w": dw}


def _places(s):
    """[E, capacity] rows of the experts, and which of them hold a slot."""
    counts = s["counts"].long()
    padded = (counts + PAD - 1) // PAD * PAD
    base = torch.cumsum(padded, 0) - padded
    i = torch.arange(s["capacity"], device=counts.device)
    return base[:, None] + i, i < counts[:, None]


def _bucket(v, at, live):
    return torch.where(live.unsqueeze(-1), v[at.clamp(max=v.shape[0] - 1)].float(), 0.0)


def _back(b, at, live, P, dtype):
    out = torch.zeros(P + 1, b.shape[2], dtype=dtype, device=b.device)
    out.index_copy_(0, torch.where(live, at, P).reshape(-1), b.to(dtype).flatten(0, 1))
    return out[:P]


def _experts(s):
    at, live = _places(s)
    P, dt, I = s["xs"].shape[0], s["xs"].dtype, s["case"]["I"]
    x, dy = _bucket(s["xs"], at, live), _bucket(s["dys"], at, live)
    W13, W2 = s["W13"].float(), s["W2"].float()
    h = x @ W13.transpose(1, 2)
    g, u = h[..., :I], h[..., I:]
    sg = torch.sigmoid(g)
    act = g * sg * u
    ys = act @ W2.transpose(1, 2)
    dact = dy @ W2
    dh = torch.cat([dact * u * sg * (1 + g * (1 - sg)), dact * g * sg], -1)
    return {"ys": _back(ys, at, live, P, dt), "dxs": _back(dh @ W13, at, live, P, dt),
            "dW13": (dh.transpose(1, 2) @ x).to(dt), "dW2": (dy.transpose(1, 2) @ act).to(dt)}


def _weight_grad(s):
    at, live = _places(s)
    return {"dW": _bucket(s["dy"], at, live).transpose(1, 2) @ _bucket(s["a"], at, live)}


def _norm(s):
    x = s["x"].float()
    r = torch.rsqrt(x.square().mean(1) + EPS)
    return {"h": (x * r.unsqueeze(1) * (s["case"]["offset"] + s["gamma"])).to(s["x"].dtype), "rstd": r}


def _norm_grad(dh, x, r, gamma, acc):
    """Gradients of x r gamma with respect to x and gamma."""
    xn = x.to(acc) * r.to(acc).unsqueeze(1)
    a = dh.to(acc) * gamma
    return r.to(acc).unsqueeze(1) * (a - xn * (a * xn).mean(1, keepdim=True)), (dh.to(acc) * xn).sum(0)


def _norm_backward(s):
    dx, dg = _norm_grad(s["dh"], s["x"], s["rstd"], s["case"]["offset"] + s["gamma"], torch.float32)
    return {"dx": (dx + s["dres"].float()).to(s["x"].dtype), "dgamma": dg}


def _join(s, acc):
    """out, its parts and the next norm; the next norm reads `out` as it is stored."""
    c = s["case"]
    y = s["y"].to(acc)
    ry = torch.rsqrt(y.square().mean(1) + EPS)
    u = y * ry.unsqueeze(1) * (c["offset"] + s["gamma"].to(acc))
    out = s["x"].to(acc) + c["scale"] * (u if s["gate"] is None else u * s["gate"].to(acc))
    out = out.to(s["x"].dtype)
    o = out.to(acc)
    ro = torch.rsqrt(o.square().mean(1) + EPS)
    return out, ry, o * ro.unsqueeze(1) * (c["offset"] + s["gamma_next"].to(acc)), ro


def _join_forward(s):
    out, ry, h, ro = _join(s, torch.float32)
    return {"out": out, "rstd_y": ry, "h": h.to(out.dtype), "rstd_out": ro}


def _join_grad(s, acc):
    c = s["case"]
    gp, gn = c["offset"] + s["gamma"].to(acc), c["offset"] + s["gamma_next"].to(acc)
    dn, dgn = _norm_grad(s["dh"], s["out"], s["rstd_out"], gn, acc)
    d = s["dres"].to(acc) + dn
    yn = s["y"].to(acc) * s["rstd_y"].to(acc).unsqueeze(1)
    v = c["scale"] * (d if s["gate"] is None else d * s["gate"].to(acc))
    b = v * gp
    dy = s["rstd_y"].to(acc).unsqueeze(1) * (b - yn * (b * yn).mean(1, keepdim=True))
    got = {"dx": d, "dy": dy, "dgamma": (v * yn).sum(0), "dgamma_next": dgn}
    if s["gate"] is not None:
        dgate = c["scale"] * d * yn * gp
        got["dgate"] = dgate.sum(0) if c["gate"] == "channel" else dgate.sum(1, keepdim=True) if c["gate"] == "token" \
            else dgate
    return got


def _join_backward(s):
    got = _join_grad(s, torch.float32)
    dt = s["x"].dtype
    return {n: v.to(dt) if n in ("dx", "dy") or (n == "dgate" and s["case"]["gate"] == "full") else v
            for n, v in got.items()}


def _route_backward(s):
    c = s["case"]
    ids, dw = s["topk_ids"].long(), s["dtopk_w"]
    if c["mode"] == 0:
        z = s["logits"] + s["logit_bias"]
        if c["renormalize"]:
            zk = z.gather(1, ids)
            p = torch.exp(zk - zk.max(1, keepdim=True).values)
            p = p / p.sum(1, keepdim=True)
            return {"dlogits": torch.zeros_like(z).scatter_(
                1, ids, c["scale"] * p * (dw - (dw * p).sum(1, keepdim=True)))}
        p = torch.exp(z - z.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
        full = torch.zeros_like(z).scatter_(1, ids, dw)
        return {"dlogits": c["scale"] * p * (full - (full * p).sum(1, keepdim=True))}
    sg = torch.sigmoid(s["logits"].gather(1, ids))
    ds = dw
    if c["renormalize"]:
        total = sg.sum(1, keepdim=True)
        ds = (dw - (dw * sg / total).sum(1, keepdim=True)) / total
    return {"dlogits": torch.zeros_like(s["logits"]).scatter_(1, ids, c["scale"] * ds * sg * (1 - sg))}


PLAIN = {"permute": _permute, "permute_backward": _permute_backward, "unpermute": _unpermute,
         "unpermute_backward": _unpermute_backward, "experts": _experts, "weight_grad": _weight_grad,
         "norm": _norm, "norm_backward": _norm_backward, "join": _join_forward, "join_backward": _join_backward,
         "route_backward": _route_backward}


# ------------------------------------------------------------------------ the framework's calls
def _own(s):
    from routing_grouped_gemm_router_gb300 import training as M
    c = s["case"]
    op = c["op"]
    if op == "permute":
        t = M.sort_tokens(s["topk_ids"], c["E"])
        xs, pos = M.permute(s["x"], s["topk_ids"], t.sorted_ids, c["E"])
        return {"xs": xs, "row_pos": pos, "sorted_ids": t.sorted_ids, "counts": t.counts}
    if op == "permute_backward":
        return {"dx": M.permute_backward(s["dxs"], s["row_pos"])}
    if op == "unpermute":
        return {"out": M.unpermute(s["ys"], s["row_pos"], s["topk_w"])}
    if op == "unpermute_backward":
        dys, dw = M.unpermute_backward(s["dout"], s["ys"], s["sorted_ids"], s["row_pos"], s["topk_w"])
        return {"dys": dys, "dtopk_w": dw}
    if op == "experts":
        h13, act = M.expert_up(s["xs"], s["W13"], s["counts"])
        ys = M.expert_down(act, s["W2"], s["counts"])
        dh13, act = M.expert_down_backward(s["dys"], s["W2"], h13, s["counts"])
        dxs = M.expert_up_backward(dh13, s["W13"], s["counts"])
        return {"ys": ys, "dxs": dxs, "dW13": M.expert_weight_grad(dh13, s["xs"], s["counts"]),
                "dW2": M.expert_weight_grad(s["dys"], act, s["counts"])}
    if op == "weight_grad":
        return {"dW": M.expert_weight_grad(s["dy"], s["a"], s["counts"], out_dtype=torch.float32)}
    if op == "norm":
        h, r = M.block_norm(s["x"], s["gamma"], eps=EPS, offset=c["offset"])
        return {"h": h, "rstd": r}
    if op == "norm_backward":
        dx, dg = M.block_norm_backward(s["dh"], s["x"], s["gamma"], s["rstd"], dres=s["dres"], offset=c["offset"])
        return {"dx": dx, "dgamma": dg}
    if op == "join":
        out, ry, h, ro = M.block_join(s["x"], s["y"], s["gamma"], gate=s["gate"], scale=c["scale"],
                                      gamma_next=s["gamma_next"], eps=EPS, offset=c["offset"])
        return {"out": out, "rstd_y": ry, "h": h, "rstd_out": ro}
    if op == "join_backward":
        g = M.block_join_backward(s["dres"], s["y"], s["gamma"], s["rstd_y"], gate=s["gate"], scale=c["scale"],
                                  dh=s["dh"], out=s["out"], gamma_next=s["gamma_next"], rstd_out=s["rstd_out"],
                                  offset=c["offset"])
        got = {"dx": g.dx, "dy": g.dy, "dgamma": g.dgamma, "dgamma_next": g.dgamma_next}
        return got if s["gate"] is None else got | {"dgate": g.dgate}
    return {"dlogits": M.route_backward(s["logits"], s["topk_ids"], s["dtopk_w"], mode=c["mode"],
                                        renormalize=c["renormalize"], scale=c["scale"],
                                        logit_bias=s["logit_bias"])}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- work and oracle
def work(case):
    c, op = case, case["op"]
    es = 2 if c.get("dtype") == "bf16" else 4
    if op == "route_backward":
        n = c["T"] * c["E"]
        dense = c["mode"] == 0 and not c["renormalize"]
        return {"bytes": 4 * n * (2 if dense else 1) + c["T"] * c["k"] * (8 if dense else 12), "flops": 4 * n}
    if op in ("norm", "norm_backward", "join", "join_backward"):
        n, full = c["T"] * c["H"], c.get("gate") == "full"
        moved = {"norm": 2, "norm_backward": 4, "join": 4 + full, "join_backward": 6 + 2 * full}[op]
        return {"bytes": moved * n * es, "flops": 10 * n}
    n = c["T"] * c["k"]
    if op == "weight_grad":
        return {"bytes": n * (c["M"] + c["N"]) * es + c["E"] * c["M"] * c["N"] * 4, "flops": 2 * n * c["M"] * c["N"]}
    if op == "experts":
        used = min(c["E"], n) * 3 * c["H"] * c["I"]  # weights that some row may need
        return {"bytes": (used + 3 * c["E"] * c["H"] * c["I"] + 4 * n * c["H"]) * es,
                "flops": 18 * n * c["H"] * c["I"]}
    tokens, rows = c["T"] * c["H"] * es, n * c["H"] * es
    moved = {"permute": tokens + rows, "permute_backward": tokens + rows, "unpermute": tokens + rows,
             "unpermute_backward": tokens + 2 * rows}[op]
    return {"bytes": moved + 8 * n, "flops": 2 * n * c["H"]}


def exact(case, seed):
    """The operators from their definitions in 64 bits, expert by expert where there are experts."""
    c, s, f = case, prepare(case, seed), torch.float64
    op = c["op"]
    if op == "permute":  # a copy: the values are the inputs'
        n = c["T"] * c["k"]
        slot = s["sorted_ids"].long()
        x = torch.cat([s["x"].to(f), torch.zeros(1, c["H"], dtype=f, device=DEV)])
        return {"xs": x[torch.where(slot < n, slot // c["k"], c["T"])], "row_pos": None, "sorted_ids": None,
                "counts": None}
    if op in ("permute_backward", "unpermute"):
        v = s["dxs" if op == "permute_backward" else "ys"]
        v = torch.cat([v, torch.zeros(1, c["H"], dtype=v.dtype, device=DEV)])
        got = torch.zeros(c["T"], c["H"], dtype=f, device=DEV)
        for j in range(c["k"]):
            w = s["topk_w"][:, j:j + 1].to(f) if op == "unpermute" else 1.0
            got += w * v[s["row_pos"][:, j].long()].to(f)  # row -1 is the zero row
        return {"dx" if op == "permute_backward" else "out": got}
    if op == "unpermute_backward":
        P = s["ys"].shape[0]
        dys = torch.zeros(P + 1, c["H"], dtype=f, device=DEV)
        dw = torch.zeros(c["T"], c["k"], dtype=f, device=DEV)
        for j in range(c["k"]):
            at = s["row_pos"][:, j].long()
            dys[torch.where(at < 0, P, at)] = s["topk_w"][:, j:j + 1].to(f) * s["dout"].to(f)
            dw[:, j] = torch.einsum("th,th->t", s["dout"].to(f), s["ys"][at.clamp(min=0)].to(f)) * (at >= 0)
        return {"dys": dys[:P], "dtopk_w": dw}
    if op == "weight_grad":
        dW = torch.zeros(c["E"], c["M"], c["N"], dtype=f, device=DEV)
        for e, r in _runs(s):
            dW[e] = s["dy"][r].to(f).T @ s["a"][r].to(f)
        return {"dW": dW}
    if op == "experts":
        P, E, H, I = s["xs"].shape[0], c["E"], c["H"], c["I"]
        got = {"ys": torch.zeros(P, H, dtype=f, device=DEV), "dxs": torch.zeros(P, H, dtype=f, device=DEV),
               "dW13": torch.zeros(E, 2 * I, H, dtype=f, device=DEV),
               "dW2": torch.zeros(E, H, I, dtype=f, device=DEV)}
        for e, r in _runs(s):
            x, dy, W13, W2 = s["xs"][r].to(f), s["dys"][r].to(f), s["W13"][e].to(f), s["W2"][e].to(f)
            g, u = x @ W13[:I].T, x @ W13[I:].T
            silu = g / (1 + torch.exp(-g))
            got["ys"][r] = (silu * u) @ W2.T
            dact = dy @ W2
            slope = (1 + torch.exp(-g) * (1 + g)) / (1 + torch.exp(-g)) ** 2  # of silu
            dg, du = dact * u * slope, dact * silu
            got["dxs"][r] = dg @ W13[:I] + du @ W13[I:]
            got["dW13"][e, :I], got["dW13"][e, I:] = dg.T @ x, du.T @ x
            got["dW2"][e] = dy.T @ (silu * u)
        return got
    if op == "norm":
        x = s["x"].to(f)
        rms = (x * x).mean(1).add(EPS).sqrt()
        return {"h": x / rms[:, None] * (c["offset"] + s["gamma"].to(f)), "rstd": 1 / rms}
    if op == "join":
        y, x = s["y"].to(f), s["x"].to(f)
        rms = (y * y).mean(1).add(EPS).sqrt()
        gate = 1.0 if s["gate"] is None else s["gate"].to(f)
        out = x + c["scale"] * gate * (y / rms[:, None]) * (c["offset"] + s["gamma"].to(f))
        o = out.to(TYPES[c["dtype"]]).to(f)  # the next norm reads what is stored
        rn = (o * o).mean(1).add(EPS).sqrt()
        return {"out": out, "rstd_y": 1 / rms, "h": o / rn[:, None] * (c["offset"] + s["gamma_next"].to(f)),
                "rstd_out": 1 / rn}
    if op == "norm_backward":
        x, dh, r = s["x"].to(f), s["dh"].to(f), s["rstd"].to(f)[:, None]
        a = dh * (c["offset"] + s["gamma"].to(f))
        along = (a * x).sum(1, keepdim=True) / c["H"]
        return {"dx": s["dres"].to(f) + r * a - r ** 3 * x * along, "dgamma": (dh * x * r).sum(0)}
    if op == "join_backward":
        y, o, dh = s["y"].to(f), s["out"].to(f), s["dh"].to(f)
        ry, ro = s["rstd_y"].to(f)[:, None], s["rstd_out"].to(f)[:, None]
        gp, gn = c["offset"] + s["gamma"].to(f), c["offset"] + s["gamma_next"].to(f)
        a = dh * gn
        d = s["dres"].to(f) + ro * a - ro ** 3 * o * (a * o).sum(1, keepdim=True) / c["H"]
        gate = torch.ones(1, 1, dtype=f, device=DEV) if s["gate"] is None else s["gate"].to(f)
        b = c["scale"] * d * gate * gp
        got = {"dx": d, "dy": ry * b - ry ** 3 * y * (b * y).sum(1, keepdim=True) / c["H"],
               "dgamma": (c["scale"] * d * gate * y * ry).sum(0), "dgamma_next": (dh * o * ro).sum(0)}
        if s["gate"] is not None:
            dgate = c["scale"] * d * y * ry * gp
            got["dgate"] = {"channel": lambda: dgate.sum(0), "token": lambda: dgate.sum(1, keepdim=True),
                            "full": lambda: dgate}[c["gate"]]()
        return got
    # the router's gradient: the derivative of the weights, one column of the Jacobian a slot
    z = s["logits"].to(f) + (s["logit_bias"].to(f) if s["logit_bias"] is not None else 0.0)
    ids = s["topk_ids"].long()
    chosen = torch.zeros_like(z).scatter_(1, ids, 1.0)
    dw = torch.zeros_like(z).scatter_(1, ids, s["dtopk_w"].to(f))
    if c["mode"] == 0:
        ex = torch.exp(z - z.amax(1, keepdim=True)) * (chosen if c["renormalize"] else 1.0)
        p = ex / ex.sum(1, keepdim=True)
        return {"dlogits": c["scale"] * (p * dw - p * (p * dw).sum(1, keepdim=True))}
    sg = chosen / (1 + torch.exp(-z))
    slope = sg * (chosen - sg)
    if not c["renormalize"]:
        return {"dlogits": c["scale"] * dw * slope}
    total = sg.sum(1, keepdim=True)
    return {"dlogits": c["scale"] * slope * (dw * total - (dw * sg).sum(1, keepdim=True)) / total ** 2}


def _runs(s):
    """(expert, its rows) for every expert that has any."""
    first, runs = 0, []
    for e, n in enumerate(s["counts"].tolist()):
        if n:
            runs.append((e, slice(first, first + n)))
        first += -(-n // PAD) * PAD
    return runs
