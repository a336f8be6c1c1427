"""The operators around a stack's blocks (embedding, layer norm, dropout and its residual join, the
router's losses) against plain 64-bit implementations, at the sizes, masks and layouts where they
can go wrong.

Tolerances are derived, not tuned. A value rounded to a type is off by at most half a step (bf16:
2^-8 of it, fp32: 2^-24 = U). A sum of n fp32 terms in any order is off by at most about n U of the
sum of their magnitudes. A row's sums have a known depth: a thread adds at most 8 chunks of 4 pairs
in turn and joins the pair, then 5 additions join a warp and 5 the warps, 43 in all and 45 with the
product by the rounded 1 / H; the tests grant 64. Magnitudes are computed in 64 bits beside the references.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
DEPTH = 64


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import _lib
    _lib.moe_device_status(True)
    return _lib


@pytest.fixture(scope="module")
def M(L):
    from routing_grouped_gemm_router_gb300 import training
    return training


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def within(got, ref, slack, what):
    """|got - ref| <= slack + half a step of got's type, everywhere."""
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = slack + HALF[got.dtype] * (ref.abs() + slack) + 1e-30
    over = (got.to(F64) - ref).abs() / bound
    assert over.max() <= 1, f"{what}: {over.max().item():.3g} times its bound"


# ------------------------------------------------------------------------------- embedding
def tokens_of(kind, g, T, V, dtype):
    if kind == "same":
        return torch.full((T,), V // 2, dtype=dtype, device=DEV)
    if kind == "outside":
        return torch.full((T,), -1, dtype=dtype, device=DEV)
    u = torch.rand(T, generator=g, device=DEV)
    t = (torch.exp(u * np.log(V + 1.0)) - 1).long().clamp(0, V - 1)
    if kind == "padded":
        t[torch.rand(T, generator=g, device=DEV) < 0.3] = -1
        t[0] = V  # just above the range
    t = t.to(dtype)
    if kind == "padded" and dtype == torch.int64 and T > 2:
        t[1], t[2] = 2 ** 32 + V // 2, -(2 ** 40)  # ids whose low 32 bits lie inside
    return t


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,V,H,kind,idt", [
    (1, 1, 8, "text", torch.int32), (1, 50000, 4096, "text", torch.int64), (7, 129280, 2880, "padded", torch.int64),
    (33, 37, 264, "padded", torch.int32), (3, 5, 72, "outside", torch.int32), (8, 32000, 7168, "text", torch.int32),
    (4099, 1000, 2056, "padded", torch.int64), (20000, 300, 512, "text", torch.int32)])
def test_embed(M, T, V, H, kind, idt, dtype):
    g = gen(T + H)
    tok = tokens_of(kind, g, T, V, idt)
    table = randn(g, V, H, dtype=dtype)
    live = (tok >= 0) & (tok < V)
    rows = torch.where(live[:, None], table[tok.clamp(0, V - 1).long()].to(F64), 0.0)
    assert torch.equal(M.embed(tok, table), rows.to(dtype))  # a copy
    scale = np.float32(45.34).item()
    within(M.embed(tok, table, scale), rows * scale, U * (rows * scale).abs(), "x")


def sums(dx, tok, V):
    """Sums of the rows of every id, their magnitudes' sums, and the ids' counts, in 64 bits."""
    live = (tok >= 0) & (tok < V)
    t, d = tok[live].long(), dx[live].to(F64)
    z = lambda *s: torch.zeros(*s, dtype=F64, device=DEV)  # noqa: E731
    n = z(V).index_add_(0, t, torch.ones(len(t), dtype=F64, device=DEV))
    return z(V, dx.shape[1]).index_add_(0, t, d), z(V, dx.shape[1]).index_add_(0, t, d.abs()), n[:, None]


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,V,H,kind,idt", [
    (1, 1, 8, "text", torch.int32), (1, 40000, 264, "text", torch.int64), (31, 3, 72, "padded", torch.int32),
    (32, 70000, 8, "text", torch.int32), (33, 5, 2056, "same", torch.int64), (64, 9, 136, "outside", torch.int32),
    (700, 511, 1000, "padded", torch.int32), (1531, 8191, 2056, "padded", torch.int64),
    (32 * 40 + 5, 300, 520, "same", torch.int32), (9001, 300000, 64, "padded", torch.int64),
    (70001, 1000, 40, "text", torch.int32), (8192, 32000, 512, "text", torch.int64)])
def test_embed_backward(M, T, V, H, kind, idt, dtype, out_dtype):
    g = gen(3 * T + V)
    tok = tokens_of(kind, g, T, V, idt)
    dx = randn(g, T, H, dtype=dtype)
    dx[(tok < 0) | (tok >= V)] = float("nan")  # padding's gradients are not read
    scale = np.float32(0.3).item()
    ref, mag, n = sums(dx, tok, V)
    slack = (n + 3) * U * scale * mag
    got = M.embed_backward(dx, tok, V, scale, out_dtype=out_dtype)
    assert got.dtype == out_dtype
    within(got, scale * ref, slack, "dtable")
    assert (got[n[:, 0] == 0] == 0).all()
    assert torch.equal(got, M.embed_backward(dx, tok, V, scale, out_dtype=out_dtype))  # the same bits
    # added to: rows of ids that do not occur are not touched
    old = randn(g, V, H, dtype=out_dtype)
    old[n[:, 0] == 0] = float("nan")
    out = old.clone()
    assert M.embed_backward(dx, tok, V, scale, out=out, accumulate=True) is out
    seen = n[:, 0] > 0
    if seen.any():
        want = old[seen].to(F64) + scale * ref[seen]
        within(out[seen], want, slack[seen] + U * want.abs(), "dtable added to")
    assert out[~seen].isnan().all()
    # and overwritten, whatever was there
    out.fill_(float("nan"))
    M.embed_backward(dx, tok, V, scale, out=out)
    assert torch.equal(out, got)


# ---------------------------------------------------------------------- layer norm, the join
def rows_of(g, T, H, dtype, kind):
    x = randn(g, T, H, std=2.0)
    if kind == "mean":  # the mean is large against the spread
        x = x * 0.01 + 100.0
    if kind == "spikes":
        x[:, ::37] *= 300.0
    return x.to(dtype)


def norm_ref(x, gamma, beta, eps):
    """h, mean, rstd in 64 bits and what each may be off by."""
    x, ga = x.to(F64), gamma.to(F64)
    be = torch.zeros_like(ga) if beta is None else beta.to(F64)
    var, mean = torch.var_mean(x, dim=1, correction=0)
    r = (var + eps).rsqrt()
    # the mean's rounding, once in a warp's own mean and once in the row's; squares of distances from
    # means that are off by dm; the reciprocal root (2 steps)
    dm = DEPTH * U * x.abs().mean(1)
    dv = (DEPTH + 6) * U * var + 4 * var.sqrt() * dm + 4 * dm ** 2
    rr = 0.51 * dv / (var + eps) + 4 * U
    xn = (x - mean[:, None]) * r[:, None]
    h = xn * ga + be
    dh = ga.abs() * (r[:, None] * dm[:, None] * (1 + rr[:, None]) + xn.abs() * (rr[:, None] + 3 * U)) \
        + 2 * U * ((xn * ga).abs() + be.abs())
    return (h, dh), (mean, dm), (r, r * rr)


SHAPES = [(1, 8), (1, 4096), (3, 72), (130, 256), (61, 264), (7, 2056), (2053, 512), (301, 2880), (40, 4104),
          (37, 7168), (9, 8200), (3, 16384), (5, 20000), (2, 32768)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_layer_norm_and_its_gradient(M, T, H, dtype):
    g = gen(T * 7 + H)
    for kind, with_beta, with_res in (("plain", True, True), ("mean", False, False), ("spikes", True, False)):
        x = rows_of(g, T, H, dtype, kind)
        gamma = 1 + randn(g, H, std=0.3)
        beta = randn(g, H, std=0.3) if with_beta else None
        eps = 1e-5
        got = M.layer_norm(x, gamma, beta, eps)
        (h, dh_), (mean, dm), (r, dr) = norm_ref(x, gamma, beta, np.float32(eps).item())
        within(got.h, h, dh_, f"h {kind}")
        within(got.mean, mean, dm, f"mean {kind}")
        within(got.rstd, r, dr, f"rstd {kind}")

        dh = randn(g, T, H, dtype=dtype)
        dres = randn(g, T, H, dtype=dtype) if with_res else None
        grads = M.layer_norm_backward(dh, x, gamma, got.mean, got.rstd, dres=dres, beta=with_beta)
        check_norm_grad(grads.dx, grads.dgamma, grads.dbeta, dh, x, gamma, got.mean, got.rstd, dres, with_beta)


def norm_grad_ref(dh, x, gamma, mean, rstd, dres):
    """dx in 64 bits from the mean and rstd that the forward pass stored, and what it may be off by."""
    dh, ga, r = dh.to(F64), gamma.to(F64), rstd.to(F64)[:, None]
    xn = (x.to(F64) - mean.to(F64)[:, None]) * r
    a = dh * ga
    s1, s2 = (a * xn).mean(1, keepdim=True), a.mean(1, keepdim=True)
    e1 = (DEPTH + 5) * U * (a * xn).abs().mean(1, keepdim=True)
    e2 = (DEPTH + 2) * U * a.abs().mean(1, keepdim=True)
    res = 0.0 if dres is None else dres.to(F64)
    dx = res + r * (a - s2 - xn * s1)
    off = r * (e2 + xn.abs() * e1) + 6 * U * ((a * r).abs() + (s2 * r).abs() + (s1 * r * xn).abs()
                                              + (0.0 if dres is None else res.abs()))
    return dx, off, xn


def check_norm_grad(dx, dgamma, dbeta, dh, x, gamma, mean, rstd, dres, with_beta):
    T = x.shape[0]
    ref, off, xn = norm_grad_ref(dh, x, gamma, mean, rstd, dres)
    within(dx, ref, off, "dx")
    prod = dh.to(F64) * xn
    within(dgamma, prod.sum(0), (T + 4) * U * prod.abs().sum(0), "dgamma")
    assert (dbeta is None) == (not with_beta)
    if with_beta:
        within(dbeta, dh.to(F64).sum(0), (T + 1) * U * dh.to(F64).abs().sum(0), "dbeta")


def test_layer_norm_of_long_batches(M):
    """More rows than the persistent CTAs take at once, and the same bits every run."""
    g = gen(5)
    T, H = 70001, 136
    x, dh = randn(g, T, H, dtype=BF), randn(g, T, H, dtype=BF)
    gamma, beta = 1 + randn(g, H, std=0.3), randn(g, H)
    got = M.layer_norm(x, gamma, beta)
    (h, slack), (mean, dm), (r, dr) = norm_ref(x, gamma, beta, np.float32(1e-5).item())
    within(got.h, h, slack, "h")
    grads = M.layer_norm_backward(dh, x, gamma, got.mean, got.rstd)
    check_norm_grad(grads.dx, grads.dgamma, grads.dbeta, dh, x, gamma, got.mean, got.rstd, None, True)
    again = M.layer_norm_backward(dh, x, gamma, got.mean, got.rstd)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_layer_norm_gradient_against_differences(M):
    """The gradient of sum(h * w) by central differences of the 64-bit formula."""
    g = gen(9)
    T, H = 3, 40
    x, w = randn(g, T, H), randn(g, T, H)
    gamma, beta = 1 + randn(g, H, std=0.3), randn(g, H)
    fwd = M.layer_norm(x, gamma, beta)
    got = M.layer_norm_backward(w, x, gamma, fwd.mean, fwd.rstd)

    def total(x, gamma, beta):
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        return (((x - mean) / (var + 1e-5).sqrt() * gamma + beta) * w.to(F64)).sum().item()

    args = [t.to(F64) for t in (x, gamma, beta)]
    for i, grad in enumerate((got.dx, got.dgamma, got.dbeta)):
        flat = grad.reshape(-1)
        for at in range(0, flat.numel(), 7):
            step = 1e-5
            up, down = [t.clone() for t in args], [t.clone() for t in args]
            up[i].reshape(-1)[at] += step
            down[i].reshape(-1)[at] -= step
            diff = (total(*up) - total(*down)) / (2 * step)
            # differences: cancellation 1e-16 * 1e2 / 1e-5 and a cubic term; the kernel: fp32 sums
            assert abs(diff - flat[at].item()) <= 1e-8 + 200 * U * max(1.0, abs(diff)) * 10


# ----------------------------------------------------------------------------------- dropout
def words(n, seed, stream, site, start=0):
    """Numbers start .. start + n - 1 of the generator, by unsigned 64-bit arithmetic (start a multiple of 4)."""
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    block = np.arange(start // 4, (start + n + 3) // 4, dtype=np.uint64)
    c = [block & low, block >> up, np.full_like(block, stream & 0xFFFFFFFF),
         np.full_like(block, ((stream >> 32) + site) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> up) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> up) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1).reshape(-1)[:n]


def test_the_generator_s_published_numbers():
    """Known answers of Philox 4x32 with 10 rounds: zeros, and all bits set."""
    assert [hex(v) for v in words(4, 0, 0, 0)] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


def factor_of(shape, p, seed, stream, site):
    """1 / (1 - p) where an element is kept, 0 where it is dropped, in 64 bits."""
    below = round(p * 2 ** 32)
    w = words(shape[0] * shape[1], seed, stream, site)
    keep = torch.from_numpy((w >= np.uint64(below)).reshape(shape)).to(DEV)
    return keep.to(F64) / (1 - below / 2 ** 32)


RNGS = [(0, 0, 0), (1234567890123456789, 41, 7), (-3, 2 ** 33 + 5, 2 ** 32 - 1), (2 ** 40 + 9, -1, 3)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 72), (1531, 2056), (37, 32768)])
def test_dropout(M, T, H, dtype):
    g = gen(T + H)
    x = randn(g, T, H, dtype=dtype)
    for (seed, stream, site), p in zip(RNGS, (0.1, 0.5, 0.999, 1e-9)):
        rng = torch.tensor([seed, stream], device=DEV)
        f = factor_of((T, H), p, seed, stream, site)
        ref = 0.7 * f * x.to(F64)
        got = M.dropout(x, p, rng, site, 0.7)
        within(got, ref, 3 * U * ref.abs(), f"dropout {p}")  # the factor, rounded, and the product
        assert (got[f == 0] == 0).all()
        assert torch.equal(got, M.dropout(x, p, rng, site, 0.7))
        bad = x.clone()
        bad[f == 0] = float("nan")  # what is dropped is not used
        assert torch.equal(got, M.dropout(bad, p, rng, site, 0.7))
    assert torch.equal(M.dropout(x, 0.0), x)


def test_dropout_keeps_the_share_it_should(M):
    """Kept elements of 2^24 with probability 0.9: within five standard deviations."""
    x = torch.ones(4096, 4096, device=DEV)
    rng = torch.tensor([5, 6], device=DEV)
    seen = [M.dropout(x, 0.1, rng, site) != 0 for site in (0, 1)]
    for kept in seen:
        assert abs(kept.double().mean().item() - 0.9) < 5 * (0.09 / 2 ** 24) ** 0.5
    both = (seen[0] & seen[1]).double().mean().item()  # two sites are independent
    assert abs(both - 0.81) < 5 * (0.81 * 0.19 / 2 ** 24) ** 0.5


def test_dropout_beyond_32_bit_offsets(M):
    """Elements behind the 2^32nd get the numbers of their own blocks."""
    T, H = (1 << 17) + 3, 32768
    x = torch.ones(T, H, dtype=BF, device=DEV)
    rng = torch.tensor([77, 1], device=DEV)
    got = M.dropout(x, 0.5, rng, 2)[-4:] != 0
    start = (T - 4) * H
    want = words(4 * H, 77, 1, 2, start) >= np.uint64(1 << 31)
    assert start > 1 << 32 or T * H > 1 << 32
    assert np.array_equal(got.cpu().numpy().reshape(-1), want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_dropout_join_and_its_gradient(M, T, H, dtype):
    g = gen(T * 5 + H)
    for p, with_beta, with_res, scale in ((0.1, True, True, 1.0), (0.0, False, True, 0.5), (0.6, True, False, 0.5)):
        x, y = randn(g, T, H, dtype=dtype, std=2.0), randn(g, T, H, dtype=dtype)
        gamma = 1 + randn(g, H, std=0.3)
        beta = randn(g, H, std=0.3) if with_beta else None
        rng = torch.tensor([17 + T, 99], device=DEV) if p else None
        f = factor_of((T, H), p, 17 + T, 99, 5) if p else torch.ones(T, H, dtype=F64, device=DEV)
        got = M.dropout_join(x, y, p, rng, 5, scale, gamma, beta, 1e-6)
        fy = scale * f * y.to(F64)
        within(got.out, x.to(F64) + fy, 3 * U * (x.to(F64).abs() + fy.abs()), "out")
        (h, dh_), (mean, dm), (r, dr) = norm_ref(got.out, gamma, beta, np.float32(1e-6).item())
        within(got.h, h, dh_, "h")
        within(got.mean, mean, dm, "mean")
        within(got.rstd, r, dr, "rstd")
        alone = M.dropout_join(x, y, p, rng, 5, scale)
        assert torch.equal(alone.out, got.out) and alone.h is None and alone.mean is None and alone.rstd is None

        dh = randn(g, T, H, dtype=dtype)
        dres = randn(g, T, H, dtype=dtype) if with_res else None
        b = M.dropout_join_backward(dres, p, rng, 5, scale, dh, got.out, gamma, got.mean, got.rstd, with_beta)
        check_norm_grad(b.dx, b.dgamma_next, b.dbeta_next, dh, got.out, gamma, got.mean, got.rstd, dres, with_beta)
        dx, off, _ = norm_grad_ref(dh, got.out, gamma, got.mean, got.rstd, dres)
        within(b.dy, scale * f * dx, scale * f * (off + 3 * U * dx.abs()), "dy")
        assert (b.dy[f == 0] == 0).all()
        if with_res:  # no next norm: dx is dres
            b = M.dropout_join_backward(dres, p, rng, 5, scale)
            assert b.dx is dres or torch.equal(b.dx, dres)
            want = scale * f * dres.to(F64)
            within(b.dy, want, 3 * U * want.abs(), "dy without a next norm")


# ------------------------------------------------------------------------- the router's losses
def balance_ref(logits, ids, mode, bias, k, offsets, mask, up):
    """Everything in 64 bits, sequence by sequence, and what losses, P and dlogits may be off by."""
    T, E = logits.shape
    bounds = [0, T] if offsets is None else offsets.tolist()
    z = logits.to(F64) + (bias.to(F64) if bias is not None and mode == 0 else 0.0)
    S = len(bounds) - 1
    take = torch.full((T,), -1, dtype=torch.long, device=DEV)
    for s in range(S):
        take[bounds[s]:bounds[s + 1]] = s
    if mask is not None:
        take[~mask] = -1
    z = torch.where((take >= 0)[:, None], z, 0.0)
    lse = torch.logsumexp(z, 1)
    soft = torch.softmax(z, 1)
    if mode == 0:
        p, slope = soft, torch.ones_like(soft)
    else:
        log_sigma = torch.nn.functional.logsigmoid(z)
        p, slope = torch.softmax(log_sigma, 1), torch.sigmoid(-z)
    # a token's probabilities: roundings of z + bias and z - max in the exponent, exponentials (2 steps
    # each), sums of at most 16 + 5 terms, quotients
    rel = U * (48 + 8 * z.abs().amax(1, keepdim=True))
    counts = torch.zeros(S, E, dtype=torch.long, device=DEV)
    prob, n = torch.zeros(S, E, dtype=F64, device=DEV), torch.zeros(S, dtype=torch.long, device=DEV)
    g, total = torch.zeros(T, E, dtype=F64, device=DEV), 0.0
    some = len({int(s) for s in take.tolist() if s >= 0})
    for s in range(S):
        rows = (take == s).nonzero()[:, 0]
        n[s] = len(rows)
        if not len(rows):
            continue
        hit = ids[rows, :k].long().reshape(-1)
        hit = hit[(hit >= 0) & (hit < E)]
        counts[s] = torch.bincount(hit, minlength=E)
        prob[s] = p[rows].mean(0)
        w = counts[s].to(F64) * E / (k * len(rows))
        total += (w * prob[s]).sum().item() / some
        g[rows] = w / (len(rows) * some)
    live = (take >= 0)[:, None]
    N = max(1, int(n.sum()))
    zl = (lse[take >= 0] ** 2).sum().item() / N
    dl = U * (30 + lse.abs() + 4 * z.abs().amax(1))  # of lse
    worst = rel[take >= 0].max().item() if live.any() else 0.0
    slack = [total * (worst + U * (int(n.max()) + E + S + 10)),
             zl * U * (N + S + 10) + (2 * lse.abs() * dl)[take >= 0].sum().item() / N]
    dot = (g * p).sum(1, keepdim=True)
    c1 = 2 * up[1].item() / N
    d = up[0].item() * p * slope * (g - dot) + c1 * lse[:, None] * soft
    off = abs(up[0].item()) * p * slope * (g + dot) * (4 * rel + 40 * U) \
        + abs(c1) * soft * (dl[:, None] + lse.abs()[:, None] * (rel + 6 * U))
    return dict(losses=torch.tensor([total, zl], dtype=F64, device=DEV),
                loss_slack=torch.tensor(slack, dtype=F64, device=DEV), counts=counts, n=n, prob=prob,
                prob_slack=prob * (worst + U * (n[:, None] + 5)), d=torch.where(live, d, 0.0),
                off=torch.where(live, off, 0.0), live=live, some=some)


CASES = [  # T, E, k, mode, offsets ("n": n random sequences), mask, spread
    (1, 1, 1, 0, None, None, 1.0), (1, 256, 8, 1, None, None, 1.0), (1, 2, 2, 0, "1", None, 1.0),
    (5, 3, 2, 1, None, "some", 1.0), (33, 7, 3, 0, "4", None, 3.0), (700, 8, 2, 0, "9", "some", 1.0),
    (700, 16, 4, 1, "300", None, 1.0), (1000, 37, 5, 1, "5", "some", 6.0), (257, 64, 6, 0, "3", None, 1.0),
    (4099, 128, 4, 0, None, "some", 2.0), (3001, 256, 8, 1, "13", None, 1.0), (513, 300, 32, 0, "2", None, 1.0),
    (129, 512, 8, 1, "7", "some", 1.0), (40, 24, 2, 0, "3", "all", 1.0), (2500, 33, 1, 1, "1", None, 30.0),
    (300, 60, 4, 0, "6", None, 40.0)]


@pytest.mark.parametrize("T,E,k,mode,seqs,masked,spread", CASES)
def test_balance_loss_and_its_gradient(M, L, T, E, k, mode, seqs, masked, spread):
    g = gen(T + 3 * E)
    logits = randn(g, T, E, std=spread) - (60 if spread > 10 and mode == 1 else 0)
    bias = randn(g, E) if E % 2 == 0 else None
    ids = logits.topk(k, 1).indices.to(torch.int32)
    shared = 2 if k < 8 else 0
    if shared:
        ids = torch.cat([ids, torch.zeros(T, shared, dtype=torch.int32, device=DEV)], 1)
    if T > 30:
        ids[torch.rand(ids.shape, generator=g, device=DEV) < 0.05] = -1
        ids[3, 0] = E
    offsets = None
    if seqs:
        S = int(seqs)
        cut = torch.randint(0, T + 1, (S + 1,), generator=g, device=DEV).sort().values.to(torch.int32)
        if S == 1:
            cut[0], cut[1] = 0, T
        offsets = cut.contiguous()  # tokens before the first and from the last on are in no sequence
    mask = None
    if masked:
        mask = torch.rand(T, generator=g, device=DEV) < 0.7
        if masked == "all":
            mask[:] = False
        mask[0] = False
    up = torch.tensor([0.7, 0.02], device=DEV)
    ref = balance_ref(logits, ids, mode, bias, k, offsets, mask, up)
    bad = logits.clone()
    bad[~ref["live"][:, 0]] = float("nan")  # what takes no part is not read
    if T > 1 and not ref["live"][0]:
        bad[0] = float("inf")
    kw = dict(mode=mode, logit_bias=bias, offsets=offsets, mask=mask)
    b = M.balance_loss(bad, ids, n_shared=shared, **kw)
    assert torch.equal(b.counts.long(), ref["counts"]) and torch.equal(b.tokens.long(), ref["n"])
    assert b.totals.tolist() == [ref["some"], int(ref["n"].sum())]
    within(b.losses, ref["losses"], ref["loss_slack"], "losses")
    within(b.prob, ref["prob"], ref["prob_slack"], "prob")
    d = M.balance_loss_backward(up, bad, b, k, **kw)
    within(d, ref["d"], ref["off"], "dlogits")
    assert (d[~ref["live"][:, 0]] == 0).all()
    old = randn(g, T, E, std=1e-3)
    out = old.clone()
    assert M.balance_loss_backward(up, bad, b, k, dlogits=out, **kw) is out
    within(out, old.to(F64) + ref["d"], ref["off"] + U * (old.to(F64) + ref["d"]).abs(), "dlogits added to")
    assert torch.equal(out[~ref["live"][:, 0]], old[~ref["live"][:, 0]])
    again = M.balance_loss(bad, ids, n_shared=shared, **kw)
    assert all(torch.equal(x, y) for x, y in zip(b, again))
    assert L.moe_device_status(True) == 0


def test_balance_of_masked_experts(M):
    """Experts whose logits are minus infinity have no probability and no gradient."""
    g = gen(4)
    for mode in (0, 1):
        logits = randn(g, 50, 12)
        logits[:, 5:9] = float("-inf")
        ids = logits.topk(3, 1).indices.to(torch.int32)
        b = M.balance_loss(logits, ids, mode=mode)
        d = M.balance_loss_backward(torch.tensor([1.0, 1.0], device=DEV), logits, b, 3, mode=mode)
        assert torch.isfinite(b.losses).all() and torch.isfinite(d).all()
        assert (b.prob[:, 5:9] == 0).all() and (d[:, 5:9] == 0).all()


def test_balance_gradient_against_differences(M):
    g = gen(6)
    T, E, k = 12, 5, 2
    offsets = torch.tensor([1, 6, 6, 11], dtype=torch.int32, device=DEV)
    for mode in (0, 1):
        logits = randn(g, T, E)
        ids = logits.topk(k, 1).indices.to(torch.int32)
        up = torch.tensor([0.8, 0.1], device=DEV)
        b = M.balance_loss(logits, ids, mode=mode, offsets=offsets)
        d = M.balance_loss_backward(up, logits, b, k, mode=mode, offsets=offsets)
        w = up.to(F64)

        def total(z):
            return (balance_ref(z, ids, mode, None, k, offsets, None, up)["losses"] * w).sum().item()

        for t in (0, 1, 5, 6, 10, 11):
            for e in range(E):
                a, c = logits.to(F64), logits.to(F64)
                a[t, e] += 1e-5
                c[t, e] -= 1e-5
                diff = (total(a) - total(c)) / 2e-5
                assert abs(diff - d[t, e].item()) <= 1e-8 + 100 * U


def test_balance_records_offsets_that_do_not_fit(M, L):
    """Offsets that decrease or leave the tokens: recorded, and nothing out of range is touched."""
    logits = randn(gen(1), 20, 8)
    ids = logits.topk(2, 1).indices.to(torch.int32)
    for off in ([0, 12, 5, 20], [-3, 10], [0, 21]):
        M.balance_loss(logits, ids, offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert L.moe_device_status(True) == 5
    M.balance_loss(logits, ids, offsets=torch.tensor([0, 20], dtype=torch.int32, device=DEV))
    assert L.moe_device_status(True) == 0


# ------------------------------------------------------------------------- graphs and streams
def test_captured_calls_and_other_streams(M):
    """All operators captured in one graph and replayed with other inputs and another stream of random
    numbers give what they give when called; so do calls on a side stream."""
    g = gen(8)
    T, H, V, E, k = 200, 264, 500, 24, 3
    tok = tokens_of("padded", g, T, V, torch.int64)
    table, y = randn(g, V, H, dtype=BF), randn(g, T, H, dtype=BF)
    gamma, beta = 1 + randn(g, H, std=0.2), randn(g, H)
    logits = randn(g, T, E)
    ids = logits.topk(k, 1).indices.to(torch.int32)
    offsets = torch.tensor([0, 20, 20, 180], dtype=torch.int32, device=DEV)
    rng = torch.tensor([3, 0], device=DEV)
    up = torch.tensor([1.0, 0.1], device=DEV)

    def all_of_them():
        x = M.dropout(M.embed(tok, table, 2.0), 0.1, rng, 0)
        n = M.layer_norm(x, gamma, beta)
        j = M.dropout_join(x, y, 0.2, rng, 1, 0.5, gamma, beta)
        b = M.balance_loss(logits, ids, offsets=offsets)
        dl = M.balance_loss_backward(up, logits, b, k, offsets=offsets)
        jb = M.dropout_join_backward(n.h, 0.2, rng, 1, 0.5, y, j.out, gamma, j.mean, j.rstd)
        nb = M.layer_norm_backward(jb.dy, x, gamma, n.mean, n.rstd, jb.dx)
        return (x, *n, *j, *b, dl, *jb, *nb, M.embed_backward(nb.dx, tok, V, 2.0, out_dtype=F32))

    all_of_them()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = all_of_them()
    for step in range(3):
        rng[1] = step
        tok.copy_(tokens_of("padded", g, T, V, torch.int64))
        logits.copy_(randn(g, T, E))
        ids.copy_(logits.topk(k, 1).indices.to(torch.int32))
        graph.replay()
        want = all_of_them()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = all_of_them()
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(other, want))
