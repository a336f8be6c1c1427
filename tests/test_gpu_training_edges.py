"""The training operators where their loops and warps take the less usual way: rows by the thousand
through the norms' rings, results that lanes of one warp store and others do not, sums next to the
ends of fp32's range. References in 64 bits; bounds are derived as in test_gpu_training."""
import pytest
import torch

from test_gpu_training import (DEV, DTYPES, F64, L, M, U, gen, randn, runs, within,  # noqa: F401
                               test_join_and_its_gradient as join_and_its_gradient)

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


# Results of M rows where M is no multiple of 32: some lanes of a warp hold rows to add to, others do not,
# while all of them load tensor memory together.
@pytest.mark.parametrize("Mm", [8, 40, 72, 136, 264, 392])
@pytest.mark.parametrize("N", [64, 136, 520])
def test_bf16_weight_gradients_added_to_by_part_of_a_warp(M, Mm, N):
    counts = [40, 0, 1, 130, 16]
    rs, P = runs(counts)
    g = gen(Mm + N)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    dy, a = randn(g, P, Mm, dtype=BF) * live, randn(g, P, N, dtype=BF) * live
    dW = randn(g, len(counts), Mm, N, dtype=BF)
    before = dW.clone()
    M.expert_weight_grad(dy, a, torch.tensor(counts, dtype=torch.int32, device=DEV), out=dW, accumulate=True)
    for e, r in rs:
        d, v = dy[r].to(F64), a[r].to(F64)
        mag = d.abs().T @ v.abs() + before[e].to(F64).abs()
        within(dW[e], before[e].to(F64) + d.T @ v, (r.stop - r.start + 3) * U * mag, BF, f"expert {e}")


def test_fp32_weight_gradients_keep_values_below_the_normal_range(M):
    """Sums and old values under 2^-126 are neither flushed on the way out nor by the addition, whether
    the tile leaves through the copy engine or from registers, in any of the kernels."""
    for dtype, Mm, N, rows in ((BF, 64, 64, 16), (F32, 64, 64, 16), (BF, 4104, 2600, 5200)):
        cnt = torch.tensor([rows], dtype=torch.int32, device=DEV)
        dy, a = torch.zeros(rows, Mm, dtype=dtype, device=DEV), torch.zeros(rows, N, dtype=dtype, device=DEV)
        dW = torch.full((1, Mm, N), 2.0 ** -133, device=DEV)
        M.expert_weight_grad(dy, a, cnt, out=dW, accumulate=True)
        assert (dW == 2.0 ** -133).all()
        dy[0], a[0] = 2.0 ** -70, 2.0 ** -62
        assert (M.expert_weight_grad(dy, a, cnt, out_dtype=F32) == 2.0 ** -132).all()
        dy[0], a[0] = 2.0 ** -60, 2.0 ** -66
        dW.fill_(-1.5 * 2.0 ** -126)
        M.expert_weight_grad(dy, a, cnt, out=dW, accumulate=True)
        assert (dW == -0.5 * 2.0 ** -126).all()


@pytest.mark.parametrize("k", [1, 3, 8])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_router_gradient_of_large_logits(M, k, renorm):
    """s (1 - s) where s is next to one: the difference may not be taken from the rounded s."""
    steps = torch.tensor([-30.0, -17.0, -8.0, -1.0, 0.0, 1.0, 8.0, 17.0, 30.0], device=DEV)
    E, T = 16, 64
    g = gen(k)
    logits = steps[torch.randint(len(steps), (T, E), generator=g, device=DEV)] + 0.5 * randn(g, T, E)
    logits[:len(steps)] = steps[:, None]  # and rows of equal ones
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1).indices
    dw = randn(g, T, k)
    z, d64 = logits.to(F64).gather(1, ids), dw.to(F64)
    s = torch.sigmoid(z)
    slope = s * torch.sigmoid(-z)
    S = s.sum(1, keepdim=True)
    want = 1.5 * slope * ((d64 - (d64 * s / S).sum(1, keepdim=True)) / S if renorm else d64)
    got = M.route_backward(logits, ids.to(torch.int32), dw, mode=1, renormalize=renorm, scale=1.5)
    # expf of an exact argument: 2 units, 4 half ones; one sum, one divide a factor; three products: 16 half units
    # with room. Renormalised, k-term sums and the quotient s / S add k + 14, to a difference of at most 2 amp
    # (relative) and to its subtrahend of at most amp: 3 k + 48
    amp = d64.abs().max(1, keepdim=True).values
    slack = 1.5 * slope * ((3 * k + 48) * U * amp / S if renorm else 16 * U * d64.abs())
    within(got.gather(1, ids), want, slack, F32, "dlogits")
    rest = torch.ones(T, E, dtype=torch.bool, device=DEV).scatter_(1, ids, False)
    assert (got[rest] == 0).all()


# Rows enough for five to dozens of units of rows a CTA, the last one ragged: stages of the ring are filled
# again and their order wraps, scalars are asked for a row ahead, column sums run over many units. Short rows
# have eight in a unit (65,541 of them: at most 8 CTAs an SM), 8200 channels of fp32 and 20,000 have no ring.
LONG = [(64, 65541), (264, 40003), (2880, 8195), (4096, 8195), (8200, 2051), (20000, 1027)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("H,T", LONG)
def test_join_and_its_gradient_over_long_batches(M, H, T, kind, dtype):
    join_and_its_gradient(M, H, T, kind, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,T", LONG)
def test_norm_and_its_gradient_over_long_batches(M, H, T, dtype):
    g, eps = gen(H + T), 1e-6
    for offset, with_res in ((0.0, True), (1.0, False)):
        x, dh, dres = (randn(g, T, H, dtype=dtype, std=2.0) for _ in range(3))
        gamma = 1 - offset + randn(g, H, std=0.3)
        h, r = M.block_norm(x, gamma, eps=eps, offset=offset)
        x64, gm, gmm, d64 = x.to(F64), offset + gamma.to(F64), offset + gamma.to(F64).abs(), dh.to(F64)
        r64 = (x64 * x64).mean(1, keepdim=True).add(eps).rsqrt()
        rel = (H / 2 + 8) * U
        within(r, r64[:, 0], rel * r64[:, 0], F32, "rstd")
        within(h, x64 * r64 * gm, (rel + 3 * U) * (x64 * r64).abs() * gmm, dtype, "h")
        dx, dg = M.block_norm_backward(dh, x, gamma, r, dres=dres if with_res else None, offset=offset)
        rk = r.to(F64)[:, None]
        a, am, xn = d64 * gm, d64.abs() * gmm, x64 * rk
        res = dres.to(F64) if with_res else torch.zeros_like(x64)
        slack = (H + 8) * U * rk * (am + xn.abs() * (am * xn.abs()).mean(1, keepdim=True)) + 2 * U * res.abs()
        within(dx, rk * (a - xn * (a * xn).mean(1, keepdim=True)) + res, slack, dtype, "dx")
        within(dg, (d64 * xn).sum(0), (T + 4) * U * (d64 * xn).abs().sum(0), F32, "dgamma")


@pytest.mark.parametrize("k", [1, 2])
def test_permute_of_copies_past_l2(M, L, k):
    """160 MB of copies: a token's row is read once for all of its slots, or, with one slot, row by row."""
    T, E, H = 20000 // k, 24, 4096
    g = gen(k)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    ids[::7, 0] = -1
    x = randn(g, T, H, dtype=BF)
    sid = M.sort_tokens(ids, E).sorted_ids
    xs, pos = M.permute(x, ids, sid, E)
    live = sid < T * k
    assert torch.equal(xs[live], x[sid[live].long() // k]) and (xs[~live] == 0).all()
    want = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    want[sid[live].long()] = torch.arange(len(sid), dtype=torch.int32, device=DEV)[live]
    assert torch.equal(pos.view(-1), want)
    assert L.moe_device_status(True) == 1  # the dropped slots


@pytest.mark.parametrize("accumulate", [False, True])
def test_fp32_weight_gradients_of_long_runs_keep_their_precision(M, accumulate):
    """The tensor cores' accumulators cut off: half a unit a step on average, always toward zero. 512 rows are
    32 steps of 16, so 32 half units of 2^-23 of the sum where the sums leave the accumulators by then, however
    long the run; over 8192 rows in one go it would be 16 times that."""
    counts = [512, 513, 0, 1023, 1024, 1040, 100, 8192, 4097]
    rs, P = runs(counts)
    g = gen(7)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    dy, a = randn(g, P, 264, dtype=BF) * live, randn(g, P, 520, dtype=BF) * live
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    dW = randn(g, len(counts), 264, 520)
    before = dW.to(F64)
    if accumulate:
        M.expert_weight_grad(dy, a, cnt, out=dW, accumulate=True)
    else:
        dW, before = M.expert_weight_grad(dy, a, cnt, out_dtype=F32), torch.zeros_like(before)
    for e, r in rs:
        want = before[e] + dy[r].to(F64).T @ a[r].to(F64)
        assert (dW[e].to(F64) - want).norm() <= 32 * 2.0 ** -24 * want.norm(), counts[e]


def off(got, want, what):
    """Sums of fp32 products, rounded as they go: a random walk of half units. Spans of 512 steps whose totals
    are added up stay below sqrt(512) of them, however long the reduction."""
    assert (got.to(F64) - want).norm() <= 512 ** 0.5 * U * want.norm(), what


@pytest.mark.parametrize("counts", [[2, 0, 31], [700, 5, 1500]])  # tiles of 32 rows, of 128
def test_fp32_products_of_long_reductions_keep_their_precision(M, counts):
    rs, P = runs(counts)
    g, long, short = gen(len(counts)), 15600, 72
    E, cnt = len(counts), torch.tensor(counts, dtype=torch.int32, device=DEV)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    # down: sums over I; the gradient of up: over 2 I; up and the gradient of down: over H
    act, dh13 = randn(g, P, long) * live, randn(g, P, long) * live
    xs, dys = randn(g, P, long) * live, randn(g, P, long) * live
    W2, W13 = randn(g, E, short, long), randn(g, E, long, short)
    U13, D2 = randn(g, E, 2 * short, long, std=long ** -0.5), randn(g, E, long, short, std=long ** -0.5)
    h13 = torch.ones(P, 2 * short, device=DEV)  # dup = dact silu(1)
    ys, dxs = M.expert_down(act, W2, cnt), M.expert_up_backward(dh13, W13, cnt)
    up, (dd, _) = M.expert_up(xs, U13, cnt)[0], M.expert_down_backward(dys, D2, h13, cnt)
    silu = torch.sigmoid(torch.ones((), dtype=F64, device=DEV))
    for e, r in rs:
        if r.start == r.stop:
            continue
        d = lambda t: t.to(F64)  # noqa: E731
        off(ys[r], d(act[r]) @ d(W2[e]).T, "ys")
        off(dxs[r], d(dh13[r]) @ d(W13[e]), "dxs")
        off(up[r], d(xs[r]) @ d(U13[e]).T, "h13")
        off(dd[r][:, short:], silu * (d(dys[r]) @ d(D2[e])), "dup")


@pytest.mark.parametrize("accumulate", [False, True])
def test_fp32_weight_gradients_of_fp32_rows_keep_their_precision(M, accumulate):
    counts = [511, 512, 513, 0, 1024, 8192, 15601]
    rs, P = runs(counts)
    g = gen(8)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    dy, a = randn(g, P, 136) * live, randn(g, P, 264) * live
    dW = randn(g, len(counts), 136, 264) if accumulate else torch.zeros(len(counts), 136, 264, device=DEV)
    before = dW.to(F64)
    M.expert_weight_grad(dy, a, torch.tensor(counts, dtype=torch.int32, device=DEV), out=dW, accumulate=accumulate)
    for e, r in rs:
        off(dW[e], before[e] + dy[r].to(F64).T @ a[r].to(F64), counts[e])
