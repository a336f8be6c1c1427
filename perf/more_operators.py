"""Cases of the operators that train a sparse stack from token ids: what each computes in plain
torch operations, and the same through the framework's training entry points.

The operators are the embedding lookup with its gradient by sorted tokens, the layer norm with
its gradient, dropout from a counter-based generator (alone, and in the residual join that also
takes the next layer norm, with its gradient), and the balance and z losses of the router with
the experts' counts and the gradient. `listed()` gives the fixed cases, `draw()` more of the
same ranges; sizes follow the workloads of `moe_inputs` (Mixtral-, gpt-oss-, Qwen3- and
DeepSeek-V3-shaped layers) or are generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the tokens of one decode step of 8 requests; latency
        dict(name="embed-few-tokens", op="embed", T=8, V=32000, H=4096, dtype="bf16", ids="int32", scale=1.0,
             outside=0.0),
        # a packed training batch with a scaled embedding, padding tokens at -1
        dict(name="embed-batch", op="embed", T=16384, V=129280, H=7168, dtype="bf16", ids="int64",
             scale=84.66, outside=0.05),
        # fp32 master gradient of the whole table from a batch of Zipf-distributed tokens
        dict(name="embed-backward-master", op="embed_backward", T=8192, V=32000, H=4096, dtype="bf16", out="f32",
             ids="int64", scale=1.0, outside=0.0),
        # an odd batch and vocabulary in fp32, with padding tokens
        dict(name="embed-backward-f32-odd", op="embed_backward", T=1531, V=8191, H=2056, dtype="f32", out="f32",
             ids="int32", scale=45.34, outside=0.1),
        # losses, counts and gradient of grouped-sigmoid routing over packed ragged sequences, padded at the end
        dict(name="balance-sequences", op="balance", T=8191, E=256, k=8, mode=1, sequences=13, masked=0.0,
             tail=0.07, bias=False),
        # the same of a softmax router over a whole batch with masked tokens
        dict(name="balance-batch", op="balance", T=32768, E=128, k=4, mode=0, sequences=0, masked=0.1,
             tail=0.0, bias=True),
        # one token's norm: latency
        dict(name="layer-norm-one-token", op="layer_norm", T=1, H=4096, dtype="bf16", beta=True),
        # the gradient in a training batch, with the residual's gradient added
        dict(name="layer-norm-backward-batch", op="layer_norm_backward", T=8192, H=7168, dtype="bf16", beta=True),
        # the same in fp32, odd sizes, no bias
        dict(name="layer-norm-backward-f32-odd", op="layer_norm_backward", T=1531, H=2056, dtype="f32",
             beta=False),
        # dropout after the embedding of an odd fp32 batch
        dict(name="dropout-f32-odd", op="dropout", T=1531, H=2056, dtype="f32", p=0.1, site=3),
        # the residual join of a training batch, with the next block's norm
        dict(name="dropout-join-batch", op="dropout_join", T=8192, H=4096, dtype="bf16", p=0.1, site=1, scale=1.0,
             beta=True),
        # its gradient, with a residual scale
        dict(name="dropout-join-backward-batch", op="dropout_join_backward", T=8192, H=4096, dtype="bf16", p=0.1,
             site=2, scale=0.5, beta=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST = 590_000_000  # bytes of a drawn case: no more than the largest listed one


def draw(rng):
    op = rng.choice(["embed", "embed_backward", "embed_backward", "balance", "balance", "balance", "layer_norm",
                     "layer_norm_backward", "layer_norm_backward", "dropout", "dropout_join",
                     "dropout_join_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "balance":
        E = _log(rng, 2, 512)
        T = min(_log(rng, 1, 32768), 4096 * 1024 // E)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 8)), mode=rng.randint(0, 1),
                    sequences=rng.choice([0, _log(rng, 1, 200)]), masked=rng.choice([0.0, 0.0, 0.2]),
                    tail=rng.choice([0.0, 0.1]), bias=rng.random() < 0.5)
    c = dict(op=op, T=_log(rng, 1, 16384), H=8 * _log(rng, 8, 896), dtype=dtype)
    if op.startswith("embed"):
        c |= dict(V=_log(rng, 256, 129280), ids=rng.choice(["int32", "int64"]), scale=rng.choice([1.0, 45.34]),
                  outside=rng.choice([0.0, 0.1]))
        if op == "embed_backward":
            c["out"] = rng.choice([dtype, "f32"])
            c["V"] = min(c["V"], 32000)
    elif op.startswith("layer_norm"):
        c["beta"] = rng.random() < 0.7
    else:
        c |= dict(p=rng.choice([0.05, 0.1, 0.5]), site=rng.randint(0, 200))
        if op != "dropout":
            c |= dict(scale=rng.choice([1.0, 0.5]), beta=rng.random() < 0.7)
    while work(c)["bytes"] > MOST:
        at = "V" if op == "embed_backward" and c["V"] > max(256, 2 * c["T"]) else "T"
        c[at] = max(1, c[at] * 3 // 4)
    return c


# ----------------------------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _tokens(c, g):
    """Token ids as text has them: the r-th most frequent about 1 / r as often as the first, some of none."""
    u = torch.rand(c["T"], generator=g, device=DEV)
    rank = (torch.exp(u * math.log(c["V"] + 1.0)) - 1.0).long().clamp(0, c["V"] - 1)
    ids = torch.randperm(c["V"], generator=g, device=DEV)[rank]
    ids[torch.rand(c["T"], generator=g, device=DEV) < c["outside"]] = -1
    return ids.to(getattr(torch, c["ids"]))


def _rows_with_mean(c, g, dt):
    """Rows as a residual stream has them: a mean of their own and a few strong channels."""
    x = _randn(g, c["T"], c["H"], std=1.5) + _randn(g, c["T"], 1, std=0.5)
    x[:, :: max(1, c["H"] // 5)] *= 8.0
    return x.to(dt)


def prepare(case, seed):
    c, s = case, {"case": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, T = c["op"], c["T"]
    if op == "balance":
        E = c["E"]
        s["logits"] = _randn(g, T, E, std=1.5) + _randn(g, E, std=0.7)
        s["logit_bias"] = _randn(g, E, std=0.5) if c["bias"] and c["mode"] == 0 else None
        key = s["logits"] if s["logit_bias"] is None else s["logits"] + s["logit_bias"]
        s["topk_ids"] = key.topk(c["k"], dim=1).indices.to(torch.int32)
        s["offsets"] = None
        if c["sequences"]:
            end = T - int(T * c["tail"])
            cuts = torch.randint(0, end + 1, (c["sequences"] - 1,), generator=g, device=DEV).sort().values
            edge = torch.tensor([0, end], device=DEV)
            s["offsets"] = torch.cat([edge[:1], cuts, edge[1:]]).to(torch.int32)
        s["mask"] = torch.rand(T, generator=g, device=DEV) >= c["masked"] if c["masked"] else None
        s["dlosses"] = _randn(g, 2).abs() + 0.01
        return s
    H, dt = c["H"], TYPES[c["dtype"]]
    if op.startswith("embed"):
        s["tokens"] = _tokens(c, g)
        if op == "embed":
            s["table"] = torch.empty(c["V"], H, dtype=dt, device=DEV)
            for v in range(0, c["V"], 8192):
                n = min(8192, c["V"] - v)
                s["table"][v:v + n] = _randn(g, n, H, dtype=dt, std=0.02)
        else:
            s["dx"] = _randn(g, T, H, dtype=dt)
        return s
    if op.startswith("dropout"):  # the generator's seed and the step's number
        s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=DEV) >> torch.tensor([0, 40], device=DEV)
    if op == "dropout":
        s["x"] = _randn(g, T, H, dtype=dt)
        return s
    s["gamma"] = 1.0 + _randn(g, H, std=0.2)
    s["beta"] = _randn(g, H, std=0.2) if c["beta"] else None
    s["x"] = _rows_with_mean(c, g, dt)
    if op == "dropout_join":
        s["y"] = _randn(g, T, H, dtype=dt)
    if op.endswith("backward"):  # x is what the norm read
        x = s["x"].double()
        mean = x.mean(1)
        s["mean"] = mean.float()
        s["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS).float()
        s["dh"] = _randn(g, T, H, dtype=dt)
        s["dres"] = _randn(g, T, H, dtype=dt)
    return s


# ------------------------------------------------------------------------------- plain forms
def _embed(s):
    tok, V = s["tokens"].long(), s["case"]["V"]
    live = (tok >= 0) & (tok < V)
    rows = s["table"][tok.clamp(0, V - 1)].float() * s["case"]["scale"]
    return {"x": torch.where(live.unsqueeze(1), rows, 0.0).to(s["table"].dtype)}


def _embed_backward(s):
    c, tok = s["case"], s["tokens"].long()
    live = (tok >= 0) & (tok < c["V"])
    d = torch.zeros(c["V"] + 1, c["H"], device=DEV)
    d.index_add_(0, torch.where(live, tok, c["V"]), s["dx"].float())
    return {"dtable": (d[:c["V"]] * c["scale"]).to(TYPES[c["out"]])}


def _layer_norm_of(x, gamma, beta):
    mean = x.mean(1)
    d = x - mean.unsqueeze(1)
    rstd = torch.rsqrt(d.square().mean(1) + EPS)
    h = d * rstd.unsqueeze(1) * gamma
    return h if beta is None else h + beta, mean, rstd


def _layer_norm(s):
    h, mean, rstd = _layer_norm_of(s["x"].float(), s["gamma"], s["beta"])
    return {"h": h.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _layer_norm_grad(s):
    """Gradients in 32 bits: dx (dres added), and the weights'."""
    dh, r = s["dh"].float(), s["rstd"].unsqueeze(1)
    xn = (s["x"].float() - s["mean"].unsqueeze(1)) * r
    a = dh * s["gamma"]
    dx = r * (a - a.mean(1, keepdim=True) - xn * (a * xn).mean(1, keepdim=True)) + s["dres"].float()
    got = {"dgamma": (dh * xn).sum(0)}
    if s["beta"] is not None:
        got["dbeta"] = dh.sum(0)
    return dx, got


def _layer_norm_backward(s):
    dx, got = _layer_norm_grad(s)
    return {"dx": dx.to(s["x"].dtype), **got}


LOW = 0xFFFFFFFF


def random_words(n, rng, site):
    """n random 32-bit numbers: Philox 4x32 with 10 rounds (Salmon et al., 2011), word i % 4 of the
    block with counter (i / 4, stream) and the seed as the key; site is added to the counter's last word."""
    seed, stream = rng[0], rng[1]
    blocks = torch.arange((n + 3) // 4, device=rng.device)
    c = [blocks & LOW, (blocks >> 32) & LOW, (stream & LOW).expand_as(blocks),
         (((stream >> 32) + site) & LOW).expand_as(blocks)]
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # the low 64 bits, whatever their sign
        c = [((b >> 32) & LOW) ^ c[1] ^ k0, b & LOW, ((a >> 32) & LOW) ^ c[3] ^ k1, a & LOW]
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack(c, 1).reshape(-1)[:n]


def _threshold(p):
    return round(p * 2.0 ** 32)  # an element is dropped where its number is below


def _mask(s):
    """1 / (1 - p) where an element is kept, 0 where it is dropped."""
    c = s["case"]
    keep = random_words(c["T"] * c["H"], s["rng"], c["site"]) >= _threshold(c["p"])
    return (keep.float() / (1.0 - _threshold(c["p"]) / 2.0 ** 32)).view(c["T"], c["H"])


def _dropout(s):
    return {"out": (s["x"].float() * _mask(s)).to(s["x"].dtype)}


def _dropout_join(s):
    out = (s["x"].float() + s["case"]["scale"] * _mask(s) * s["y"].float()).to(s["x"].dtype)
    h, mean, rstd = _layer_norm_of(out.float(), s["gamma"], s["beta"])  # the norm reads what is stored
    return {"out": out, "h": h.to(out.dtype), "mean": mean, "rstd": rstd}


def _dropout_join_backward(s):
    dx, got = _layer_norm_grad(s)
    dt = s["x"].dtype
    return {"dx": dx.to(dt), "dy": (s["case"]["scale"] * _mask(s) * dx).to(dt), **got}


def _sequence(s):
    """Sequence of every token, -1 for tokens that take no part, and how many sequences there are."""
    T, off = s["case"]["T"], s["offsets"]
    t = torch.arange(T, device=DEV)
    if off is None:
        seq, S = torch.zeros(T, dtype=torch.long, device=DEV), 1
    else:
        S = off.numel() - 1
        seq = torch.searchsorted(off.long(), t, right=True) - 1
        seq = torch.where(seq < S, seq, -1)
    if s["mask"] is not None:
        seq = torch.where(s["mask"], seq, -1)
    return seq, S


def _balance(s):
    """Losses, counts, live tokens and mean probabilities a sequence, and the gradient of the losses."""
    c = s["case"]
    seq, S = _sequence(s)
    live = seq >= 0
    z = s["logits"] if s["logit_bias"] is None else s["logits"] + s["logit_bias"]
    top = z.max(1, keepdim=True).values
    ex = torch.exp(z - top)
    total = ex.sum(1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    if c["mode"] == 0:
        p = ex / total
    else:
        p = torch.sigmoid(z)
        p = p / p.sum(1, keepdim=True)
    at = torch.where(live, seq, S)
    n = torch.zeros(S + 1, device=DEV).index_add_(0, at, torch.ones_like(lse))[:S]
    counts = torch.zeros((S + 1) * c["E"], dtype=torch.int32, device=DEV)
    slot = (at.unsqueeze(1) * c["E"] + s["topk_ids"].long()).reshape(-1)
    counts.index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    counts = counts.view(S + 1, c["E"])[:S]
    P = torch.zeros(S + 1, c["E"], device=DEV).index_add_(0, at, p)[:S] / n.clamp(min=1).unsqueeze(1)
    f = counts * (c["E"] / c["k"]) / n.clamp(min=1).unsqueeze(1)
    nonempty = (n > 0).sum().clamp(min=1)
    tokens = n.sum().clamp(min=1)
    losses = torch.stack([(f * P).sum() / nonempty, torch.where(live, lse * lse, 0.0).sum() / tokens])
    at = seq.clamp(min=0)
    g = f[at] / (n[at].clamp(min=1) * nonempty).unsqueeze(1)  # of the balance loss, to p
    dz = p * (g - (g * p).sum(1, keepdim=True))
    soft = p
    if c["mode"] == 1:
        dz = dz * torch.sigmoid(-z)
        soft = torch.softmax(z, 1)
    dz = s["dlosses"][0] * dz + s["dlosses"][1] * 2.0 / tokens * lse.unsqueeze(1) * soft
    return {"losses": losses, "counts": counts, "tokens": n.to(torch.int32), "prob": P,
            "dlogits": torch.where(live.unsqueeze(1), dz, 0.0)}


PLAIN = {"embed": _embed, "embed_backward": _embed_backward, "layer_norm": _layer_norm,
         "layer_norm_backward": _layer_norm_backward, "dropout": _dropout, "dropout_join": _dropout_join,
         "dropout_join_backward": _dropout_join_backward, "balance": _balance}


# ------------------------------------------------------------------------ the framework's calls
def _own(s):
    from routing_grouped_gemm_router_gb300 import training as M
    c = s["case"]
    op = c["op"]
    if op == "embed":
        return {"x": M.embed(s["tokens"], s["table"], scale=c["scale"])}
    if op == "embed_backward":
        return {"dtable": M.embed_backward(s["dx"], s["tokens"], c["V"], scale=c["scale"],
                                           out_dtype=TYPES[c["out"]])}
    if op == "layer_norm":
        return M.layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS)._asdict()
    if op == "layer_norm_backward":
        g = M.layer_norm_backward(s["dh"], s["x"], s["gamma"], s["mean"], s["rstd"], dres=s["dres"],
                                  beta=s["beta"] is not None)
        return {n: v for n, v in g._asdict().items() if v is not None}
    if op == "dropout":
        return {"out": M.dropout(s["x"], c["p"], s["rng"], site=c["site"])}
    if op == "dropout_join":
        return M.dropout_join(s["x"], s["y"], c["p"], s["rng"], site=c["site"], scale=c["scale"],
                              gamma_next=s["gamma"], beta_next=s["beta"], eps=EPS)._asdict()
    if op == "dropout_join_backward":
        g = M.dropout_join_backward(s["dres"], c["p"], s["rng"], site=c["site"], scale=c["scale"], dh=s["dh"],
                                    out=s["x"], gamma_next=s["gamma"], mean=s["mean"], rstd=s["rstd"],
                                    beta=s["beta"] is not None)
        got = {"dx": g.dx, "dy": g.dy, "dgamma": g.dgamma_next}
        return got if g.dbeta_next is None else got | {"dbeta": g.dbeta_next}
    how = dict(mode=c["mode"], logit_bias=s["logit_bias"], offsets=s["offsets"], mask=s["mask"])
    b = M.balance_loss(s["logits"], s["topk_ids"], **how)
    return {"losses": b.losses, "counts": b.counts, "tokens": b.tokens, "prob": b.prob,
            "dlogits": M.balance_loss_backward(s["dlosses"], s["logits"], b, c["k"], **how)}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- work and oracle
def work(case):
    c, op, T = case, case["op"], case["T"]
    if op == "balance":
        n = T * c["E"]
        return {"bytes": 8 * n + 4 * T * c["k"], "flops": 18 * n}
    es = 2 if c["dtype"] == "bf16" else 4
    n = T * c["H"]
    ids = T * (8 if c.get("ids") == "int64" else 4)
    if op == "embed":  # a row is read once, however many tokens share it
        return {"bytes": (n + min(T, c["V"]) * c["H"]) * es + ids, "flops": n}
    if op == "embed_backward":
        return {"bytes": n * es + c["V"] * c["H"] * (2 if c["out"] == "bf16" else 4) + ids, "flops": n}
    moved = {"layer_norm": 2, "layer_norm_backward": 4, "dropout": 2, "dropout_join": 4, "dropout_join_backward": 5}
    return {"bytes": moved[op] * n * es, "flops": 12 * n}


def _numpy_keep(c, rng):
    """The kept elements by 64-bit unsigned arithmetic on the host."""
    seed, stream = (int(v) for v in rng.tolist())
    n = c["T"] * c["H"]
    block = np.arange(-(-n // 4), dtype=np.uint64)
    low, up = np.uint64(LOW), np.uint64(32)
    x0, x1 = block & low, block >> up
    x2 = np.full_like(block, stream & LOW)
    x3 = np.full_like(block, ((stream >> 32) + c["site"]) & LOW)
    key = [seed & LOW, seed >> 32 & LOW]
    for r in range(10):
        q0, q1 = (np.uint64((k + r * w) & LOW) for k, w in zip(key, (0x9E3779B9, 0xBB67AE85)))
        m0, m1 = np.uint64(0xD2511F53) * x0, np.uint64(0xCD9E8D57) * x2
        x0, x1, x2, x3 = (m1 >> up) ^ x1 ^ q0, m1 & low, (m0 >> up) ^ x3 ^ q1, m0 & low
    kept = np.empty((block.size, 4), dtype=bool)
    for i, w in enumerate((x0, x1, x2, x3)):
        kept[:, i] = w >= np.uint64(_threshold(c["p"]))
    return torch.from_numpy(kept.reshape(-1)[:n].reshape(c["T"], c["H"])).to(DEV)


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    c, s, f = case, prepare(case, seed), torch.float64
    op = c["op"]
    if op == "embed":
        table = torch.cat([s["table"], torch.zeros(1, c["H"], dtype=s["table"].dtype, device=DEV)])
        return {"x": table[s["tokens"].long()].to(f) * c["scale"]}  # token -1 is the row of zeros
    if op == "embed_backward":
        d = torch.zeros(c["V"], c["H"], dtype=f, device=DEV)
        tok, order = s["tokens"].long().sort(stable=True)
        seen, counts = tok.unique_consecutive(return_counts=True)
        ends = counts.cumsum(0).tolist()
        first = 0
        for v, end in zip(seen.tolist(), ends):
            if v >= 0:
                d[v] = s["dx"][order[first:end]].to(f).sum(0) * c["scale"]
            first = end
        return {"dtable": d}
    if op == "balance":
        return _exact_balance(c, s)
    factor = None
    if op.startswith("dropout"):
        factor = _numpy_keep(c, s["rng"]).to(f) * (2.0 ** 32 / (2.0 ** 32 - _threshold(c["p"])))
    if op == "dropout":
        return {"out": s["x"].to(f) * factor}
    gamma = s["gamma"].to(f)
    got = {}
    x = s["x"].to(f)
    if op in ("layer_norm", "dropout_join"):
        if op == "dropout_join":
            got["out"] = x + c["scale"] * factor * s["y"].to(f)
            x = got["out"].to(s["x"].dtype).to(f)  # the next norm reads what is stored
        var, mean = torch.var_mean(x, dim=1, correction=0)
        h = gamma * (x - mean[:, None]) / (var + EPS).sqrt()[:, None]
        return got | {"h": h if s["beta"] is None else h + s["beta"].to(f), "mean": mean,
                      "rstd": 1 / (var + EPS).sqrt()}
    dh, r, H = s["dh"].to(f), s["rstd"].to(f)[:, None], c["H"]
    off = x - s["mean"].to(f)[:, None]
    a = dh * gamma
    got["dx"] = s["dres"].to(f) + r * a - r * a.sum(1, keepdim=True) / H \
        - r ** 3 * off * (a * off).sum(1, keepdim=True) / H
    if factor is not None:
        got["dy"] = got["dx"] * factor * c["scale"]
    got["dgamma"] = torch.einsum("th,th,t->h", dh, off, r[:, 0])
    if s["beta"] is not None:
        got["dbeta"] = dh.sum(0)
    return got


def _exact_balance(c, s):
    """Sequence by sequence, with the gradient as a product with the Jacobian's parts."""
    f, E, T = torch.float64, c["E"], c["T"]
    bounds = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    S = len(bounds) - 1
    here = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    z = s["logits"].to(f) + (0.0 if s["logit_bias"] is None else s["logit_bias"].to(f))
    lse = torch.logsumexp(z, 1)
    raw = torch.exp(z) if c["mode"] == 0 else 1 / (1 + torch.exp(-z))
    share = raw / raw.sum(1, keepdim=True)
    slope = share if c["mode"] == 0 else share / (1 + torch.exp(z))
    prob, losses = torch.zeros(S, E, dtype=f, device=DEV), torch.zeros(2, dtype=f, device=DEV)
    dbal = torch.zeros(T, E, dtype=f, device=DEV)
    taking, nonempty = torch.zeros(T, dtype=torch.bool, device=DEV), 0
    for q, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        rows = torch.arange(a, b, device=DEV)[here[a:b]]
        n = rows.numel()
        if not n:
            continue
        nonempty += 1
        taking[rows] = True
        hits = torch.bincount(s["topk_ids"][rows].long().reshape(-1), minlength=E).to(f)
        prob[q] = share[rows].mean(0)
        w = hits * E / (c["k"] * n)
        losses[0] += (w * prob[q]).sum()
        dbal[rows] = slope[rows] * (w - share[rows] @ w[:, None]) / n
    many = int(taking.sum())
    losses[0] /= max(1, nonempty)
    losses[1] = lse[taking].square().sum() / max(1, many)
    dz = 2 * lse[:, None] * torch.exp(z - lse[:, None]) * taking[:, None] / max(1, many)
    up = s["dlosses"].to(f)
    return {"losses": losses, "counts": None, "tokens": None, "prob": prob,
            "dlogits": up[0] * dbal / max(1, nonempty) + up[1] * dz}
