"""The training operators against plain 64-bit implementations, at the sizes, masks and layouts
where they can go wrong.

Tolerances are derived, not tuned. A value rounded to a type is off by at most half a step
(bf16: 2^-8 of it, fp32: 2^-24). A sum of n fp32 products in any order is off by at most about
n * 2^-24 of the sum of the products' magnitudes; each bound below adds the few roundings of
the arithmetic around the sum. Magnitudes are computed in 64 bits beside the references.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24  # half a step of fp32
DTYPES = [torch.bfloat16, torch.float32]


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


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def within(got, ref, slack, dtype, what):
    """|got - ref| <= slack + half a step of dtype, everywhere."""
    assert got.dtype == dtype and got.shape == ref.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = slack + HALF[dtype] * (ref.abs() + slack) + 1e-30
    over = (got.to(F64) - ref).abs() / bound
    assert over.max() <= 1, f"{what}: {over.max().item():.3g} times its bound"


# -------------------------------------------------------------------------------- dispatch
def random_ids(g, T, k, E, drop):
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    if drop == "some":
        ids[torch.rand(T, k, generator=g, device=DEV) < 0.3] = -1
        ids[0, 0] = E + 5  # above the range too
    if drop == "all":
        ids[:] = -1
    return ids


def table(ids, E, P):
    """The expert-sorted rows by a loop over slots: (sorted_ids, row_pos, counts)."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    sid, pos, counts, at = [T * k] * P, [-1] * (T * k), [], 0
    for e in range(E):
        slots = [r for r, v in enumerate(flat) if v == e]
        for i, r in enumerate(slots):
            sid[at + i], pos[r] = r, at + i
        counts.append(len(slots))
        at += -(-len(slots) // 16) * 16
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return t(sid), t(pos).view(T, k), t(counts)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,drop", [
    (1, 1, 1, 8, None), (1, 4, 128, 2880, None), (7, 3, 5, 264, "some"), (3, 2, 4, 64, "all"),
    (33, 32, 40, 72, "some"), (4099, 5, 24, 3400, "some"), (130, 2, 300, 1000, None), (5, 2, 8, 8200, None), (700, 8, 64, 128, "some")])
def test_dispatch_and_its_gradients(M, L, T, k, E, H, drop, dtype):
    g = gen(T * 31 + H)
    ids = random_ids(g, T, k, E, drop)
    P = M.buffer_rows(T, k, E)
    sid, pos, counts = table(ids, E, P)
    t = M.sort_tokens(ids, E)
    assert torch.equal(t.sorted_ids, sid) and torch.equal(t.counts, counts)
    x = randn(g, T, H, dtype=dtype)
    xs, got_pos = M.permute(x, ids, t.sorted_ids, E)
    assert torch.equal(got_pos, pos)
    live = sid < T * k
    want = torch.zeros(P, H, dtype=dtype, device=DEV)
    want[live] = x[sid[live].long() // k]
    assert torch.equal(xs, want)  # a copy: bit for bit, zeros elsewhere

    # rows of no slot hold NaN: nothing may read them
    ys = randn(g, P, H, dtype=dtype)
    ys[~live] = float("nan")
    w = torch.rand(T, k, generator=g, device=DEV)
    kept = (pos >= 0).unsqueeze(-1)
    rows = torch.where(kept, ys[pos.clamp(min=0).long()].to(F64), 0.0)
    for weighted in (False, True):
        f = w.to(F64).unsqueeze(-1) if weighted else torch.ones(T, k, 1, dtype=F64, device=DEV)
        got = M.unpermute(ys, pos, w) if weighted else M.permute_backward(ys, pos)
        within(got, (f * rows).sum(1), (k + 2) * U * (f * rows).abs().sum(1), dtype, f"slot sum, weighted {weighted}")

    dout = randn(g, T, H, dtype=dtype)
    dys, dw = M.unpermute_backward(dout, ys, sid, pos, w)
    want = torch.zeros(P, H, dtype=F64, device=DEV)
    s = sid[live].long()
    want[live] = w.to(F64).reshape(-1)[s, None] * dout.to(F64)[s // k]
    within(dys, want, U * want.abs(), dtype, "dys")
    assert (dys[~live] == 0).all()
    prod = rows * dout.to(F64).unsqueeze(1)
    within(dw, prod.sum(-1), (H + 2) * U * prod.abs().sum(-1), torch.float32, "dtopk_w")
    assert (dw[pos < 0] == 0).all()
    assert L.moe_device_status(True) == (1 if drop else 0)  # the align step records dropped ids


def test_dispatch_positions_outside_the_buffer_count_as_dropped(M, L):
    T, k, H, P = 4, 2, 64, 32
    g = gen(3)
    pos = torch.tensor([[0, 99], [-7, 31], [1 << 30, 2], [3, 32]], dtype=torch.int32, device=DEV)
    sid = torch.full((P,), T * k, dtype=torch.int32, device=DEV)
    sid[5], sid[6] = -3, 1 << 30
    ys, w, dout = randn(g, P, H), torch.rand(T, k, generator=g, device=DEV), randn(g, T, H)
    ok = ((pos >= 0) & (pos < P)).unsqueeze(-1)
    rows = torch.where(ok, ys[pos.clamp(0, P - 1).long()].to(F64), 0.0)
    want = (rows * w.to(F64).unsqueeze(-1)).sum(1)
    within(M.unpermute(ys, pos, w), want, 4 * U * (rows * w.unsqueeze(-1)).abs().sum(1), torch.float32, "out")
    dys, dw = M.unpermute_backward(dout, ys, sid, pos, w)
    assert (dw[~ok.squeeze(-1)] == 0).all() and torch.isfinite(dw).all()
    ids = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    xs, _ = M.permute(dout, ids, sid, 4)
    assert (xs == 0).all()


# --------------------------------------------------------------------------------- experts
COUNTS = {
    "one": [1],
    "edges": [0, 1, 15, 16, 17, 0, 127, 128, 129, 0],
    "long": [300, 0, 5, 513],
    "empty": [0, 0, 0],
    "many": [(7 * e) % 23 for e in range(70)],
    "first-last": [0] * 30 + [40] + [0] * 33 + [3],
    # enough rows for the tensor-core kernels' wide items, which long dimensions below then take
    "wide": [257, 0, 300, 1000, 17, 700],
}


def runs(counts):
    at, out = 0, []
    for e, n in enumerate(counts):
        out.append((e, slice(at, at + n)))
        at += -(-n // 16) * 16
    return out, at


def expert_inputs(name, H, I, dtype, seed):
    """Rows, weights and gradients of a layout; the tail past the last run is two blocks and a bit."""
    counts = COUNTS[name]
    rs, end = runs(counts)
    P, E, g = end + 48, len(counts), gen(seed)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    xs, dys = (randn(g, P, H, dtype=dtype) * live for _ in range(2))
    W13 = randn(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5)
    W2 = randn(g, E, H, I, dtype=dtype, std=I ** -0.5)
    return counts, rs, live, xs, dys, W13, W2, torch.tensor(counts, dtype=torch.int32, device=DEV)


EXPERT_SHAPES = [("one", 8, 8), ("edges", 64, 96), ("edges", 264, 520), ("long", 320, 136), ("empty", 64, 64),
                 ("many", 136, 72), ("first-last", 1032, 256), ("long", 512, 768), ("wide", 4104, 6600),
                 ("wide", 13000, 2056)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name,H,I", EXPERT_SHAPES)
def test_expert_products_and_gradients(M, L, name, H, I, dtype):
    counts, rs, live, xs, dys, W13, W2, cnt = expert_inputs(name, H, I, dtype, H + I)
    P, E, half = xs.shape[0], len(counts), HALF[dtype]
    x64, dy64 = xs.to(F64), dys.to(F64)
    h13, act = M.expert_up(xs, W13, cnt)
    ys = M.expert_down(act, W2, cnt)
    dh13, act2 = M.expert_down_backward(dys, W2, h13, cnt)
    dxs = M.expert_up_backward(dh13, W13, cnt)
    dW2, dW13 = M.expert_weight_grad(dys, act2, cnt), M.expert_weight_grad(dh13, xs, cnt)
    for v in (h13, act, ys, dh13, act2, dxs):
        assert (v[~live.squeeze(1)] == 0).all()  # rows of no slot
    a64, h64, dh64 = act.to(F64), h13.to(F64), dh13.to(F64)
    f32 = torch.float32
    for e, r in rs:
        if r.start == r.stop:
            assert (dW2[e] == 0).all() and (dW13[e] == 0).all()
            continue
        w13, w2 = W13[e].to(F64), W2[e].to(F64)
        # each product from the operands that the kernel read
        hm = x64[r].abs() @ w13.abs().T
        within(h13[r], x64[r] @ w13.T, (H + 2) * U * hm, f32, "h13")
        # silu from h13; expf and the divide: a few units of fp32 (8 here), and an error of h13 within a
        # step of what was stored moves silu by at most its slope, below 1.1
        g_, u_ = h64[r, :I], h64[r, I:]
        s = torch.sigmoid(g_)
        silu = g_ * s
        within(act[r], silu * u_, 16 * U * ((g_ * u_).abs() + hm[:, :I] + hm[:, I:] * 1e-30), dtype, "act")
        assert torch.equal(act[r], act2[r])
        within(ys[r], a64[r] @ w2.T, (I + 2) * U * (a64[r].abs() @ w2.abs().T), dtype, "ys")
        dact, dm = dy64[r] @ w2, dy64[r].abs() @ w2.abs()
        slope = s * (1 + g_ * (1 - s))
        within(dh13[r, :I], dact * u_ * slope, (H + 24) * U * dm * u_.abs() * (1 + g_.abs()), dtype, "dgate")
        within(dh13[r, I:], dact * silu, (H + 24) * U * dm * g_.abs(), dtype, "dup")
        within(dxs[r], dh64[r] @ w13, (2 * I + 2) * U * (dh64[r].abs() @ w13.abs()), dtype, "dxs")
        n = r.stop - r.start
        within(dW2[e], dy64[r].T @ a64[r], (n + 2) * U * (dy64[r].abs().T @ a64[r].abs()), dtype, "dW2")
        within(dW13[e], dh64[r].T @ x64[r], (n + 2) * U * (dh64[r].abs().T @ x64[r].abs()), dtype, "dW13")
    assert L.moe_device_status(True) == 0


# Several rounds of 256-column tiles over the CTA pairs, the last one more or less than half full, with
# many short runs of rows.
@pytest.mark.parametrize("H,I", [(264, 520), (520, 264), (1000, 1000)])
def test_expert_products_over_several_rounds_of_tiles(M, L, H, I):
    test_expert_products_and_gradients(M, L, "many", H, I, torch.bfloat16)


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.float32, torch.float32)])
@pytest.mark.parametrize("Mm,N", [(72, 200), (256, 256), (520, 264), (4104, 2600)])
def test_weight_grad_accumulates(M, Mm, N, dtype, out):
    # the last size takes the wide items, with a last item of one tile and an expert without rows
    counts = [2600, 0, 5200] if N > 1000 else COUNTS["edges"] + [700]
    rs, P = runs(counts)
    g = gen(Mm)
    live = torch.zeros(P, 1, dtype=torch.bool, device=DEV)
    for _, r in rs:
        live[r] = True
    dy, a = randn(g, P, Mm, dtype=dtype) * live, randn(g, P, N, dtype=dtype) * live
    cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
    dW = randn(g, len(counts), Mm, N, dtype=out)
    before = dW.clone()
    got = M.expert_weight_grad(dy, a, cnt, out=dW, accumulate=True)
    assert got is dW
    for e, r in rs:
        d, v = dy[r].to(F64), a[r].to(F64)
        ref = before[e].to(F64) + d.T @ v
        mag = d.abs().T @ v.abs() + before[e].to(F64).abs()
        within(dW[e], ref, (r.stop - r.start + 3) * U * mag, out, f"expert {e}")
        if r.start == r.stop:
            assert torch.equal(dW[e], before[e])
    fresh = M.expert_weight_grad(dy, a, cnt, out_dtype=out)
    over = M.expert_weight_grad(dy, a, cnt, out=torch.full_like(dW, float("nan")))
    assert torch.equal(fresh, over)  # overwritten, and the same bits every time


def test_counts_that_do_not_fit_are_cut(M, L):
    H = I = 64
    g, P = gen(1), 64
    xs, W13 = randn(g, P, H, dtype=torch.bfloat16), randn(g, 4, 2 * I, H, dtype=torch.bfloat16)
    for counts in ([40, 40, 40, 40], [-5, 10, 1 << 30, 3], [70, 0, 0, 0]):
        cnt = torch.tensor(counts, dtype=torch.int32, device=DEV)
        _, act = M.expert_up(xs, W13, cnt)
        M.expert_weight_grad(xs, act, cnt)
        torch.cuda.synchronize()
        assert L.moe_device_status(True) == 4


def test_infinite_and_nan_rows_stay_in_their_expert(M):
    """A row that overflowed must not reach another expert's results."""
    for dtype in DTYPES:
        counts, rs, live, xs, dys, W13, W2, cnt = expert_inputs("edges", 264, 136, dtype, 9)
        bad = rs[4][1]  # expert 4, between others in the same tiles
        ref = M.expert_up(xs, W13, cnt) + (M.expert_weight_grad(dys, xs, cnt),)
        xs[bad.start], xs[bad.start + 1] = float("inf"), float("nan")
        h13, act = M.expert_up(xs, W13, cnt)
        dW = M.expert_weight_grad(dys, xs, cnt)
        keep = torch.ones(xs.shape[0], dtype=torch.bool, device=DEV)
        keep[bad] = False
        assert torch.equal(h13[keep], ref[0][keep]) and torch.equal(act[keep], ref[1][keep])
        others = [e for e in range(len(counts)) if e != 4]
        assert torch.equal(dW[others], ref[2][others])
        assert torch.isnan(dW[4]).any()


# ------------------------------------------------------------------------------------ norms
def gate_of(g, kind, T, H, dtype):
    if kind == "none":
        return None
    shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}[kind]
    return torch.sigmoid(randn(g, *shape)).to(dtype if kind == "full" else torch.float32)


def join64(x, y, gamma, gate, scale, gamma_next, eps, offset, dtype, rounding=None):
    """The join in 64 bits; the next norm reads `out` plus `rounding` (what storing it added)."""
    ry = (y * y).mean(1, keepdim=True).add(eps).rsqrt()
    out = x + scale * (1.0 if gate is None else gate) * (y * ry * (offset + gamma))
    if gamma_next is None:
        return out, ry, None, None
    o = out if rounding is None else out + rounding
    ro = (o * o).mean(1, keepdim=True).add(eps).rsqrt()
    return out, ry, o * ro * (offset + gamma_next), ro


NORM_H = [8, 64, 264, 1000, 2880, 8192, 8200, 16384, 16392, 32768]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", NORM_H)
def test_norm_and_its_gradient(M, H, dtype):
    for T, offset, with_res in ((1, 0.0, True), (5, 1.0, False), (307, 0.0, True)):
        g, eps = gen(H + T), 1e-6
        x, dh, dres = (randn(g, T, H, dtype=dtype, std=2.0) for _ in range(3))
        x[T // 2] = 0  # rstd = eps^-1/2: large, finite
        gamma = 1 - offset + randn(g, H, std=0.3)
        h, r = M.block_norm(x, gamma, eps=eps, offset=offset)
        x64, gm, d64 = x.to(F64), offset + gamma.to(F64), dh.to(F64)
        r64 = (x64 * x64).mean(1, keepdim=True).add(eps).rsqrt()
        # sum of squares: H terms of one sign; rsqrt a few units: relative (H + 8) / 2 units at most
        rel = (H / 2 + 8) * U
        within(r, r64[:, 0], rel * r64[:, 0], torch.float32, "rstd")
        within(h, x64 * r64 * gm, (rel + 3 * U) * (x64 * r64).abs() * (offset + gamma.to(F64).abs()), dtype, "h")
        dx, dg = M.block_norm_backward(dh, x, gamma, r, dres=dres if with_res else None, offset=offset)
        rk = r.to(F64)[:, None]  # the kernel's own rstd is an input of the backward pass
        a, xn = d64 * gm, x64 * rk
        am = d64.abs() * (offset + gamma.to(F64).abs())
        m = (a * xn).mean(1, keepdim=True)
        slack = (H + 8) * U * rk * (am + xn.abs() * (am * xn.abs()).mean(1, keepdim=True))
        res = dres.to(F64) if with_res else torch.zeros_like(x64)
        within(dx, rk * (a - xn * m) + res, slack + 2 * U * res.abs(), dtype, "dx")
        within(dg, (d64 * xn).sum(0), (T + 4) * U * (d64 * xn).abs().sum(0), torch.float32, "dgamma")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("H,T", [(8, 1), (264, 37), (2880, 301), (8200, 5), (20000, 3)])
def test_join_and_its_gradient(M, H, T, kind, dtype):
    for nxt, with_res, scale, offset in ((True, True, 0.5, 1.0), (True, False, 1.0, 0.0), (False, True, -2.0, 0.0)):
        g, eps = gen(H * 7 + T), 1e-6
        x, y, dres, dh = (randn(g, T, H, dtype=dtype) for _ in range(4))
        gamma, gamma_next = (1 - offset + randn(g, H, std=0.3) for _ in range(2))
        gate = gate_of(g, kind, T, H, dtype)
        j = M.block_join(x, y, gamma, gate=gate, scale=scale, gamma_next=gamma_next if nxt else None, eps=eps,
                         offset=offset)
        up = lambda t: None if t is None else t.to(F64)  # noqa: E731
        x64, y64, ga, gn, gt = up(x), up(y), up(gamma), up(gamma_next), up(gate)
        out64, ry, _, _ = join64(x64, y64, ga, gt, scale, None, eps, offset, dtype)
        rel = (H / 2 + 8) * U
        within(j.rstd_y, ry[:, 0], rel * ry[:, 0], torch.float32, "rstd_y")
        part = (out64 - x64).abs()
        within(j.out, out64, (rel + 6 * U) * (part + (scale * (1.0 if gt is None else gt) * y64 * ry).abs()
                                              * (offset + ga.abs())) + U * x64.abs(), dtype, "out")
        o64 = up(j.out)
        if nxt:
            ro = (o64 * o64).mean(1, keepdim=True).add(eps).rsqrt()
            within(j.rstd_out, ro[:, 0], rel * ro[:, 0], torch.float32, "rstd_out")
            within(j.h, o64 * ro * (offset + gn), (rel + 3 * U) * (o64 * ro).abs() * (offset + gn.abs()), dtype, "h")
        else:
            assert j.h is None and j.rstd_out is None
        b = M.block_join_backward(dres if with_res else None, y, gamma, j.rstd_y, gate=gate, scale=scale,
                                  offset=offset, **(dict(dh=dh, out=j.out, gamma_next=gamma_next,
                                                         rstd_out=j.rstd_out) if nxt else {}))
        # in 64 bits from what the backward pass was given; *_m are magnitudes of the terms
        d = dm = torch.zeros_like(x64)
        if with_res:
            d, dm = up(dres), up(dres).abs()
        if nxt:
            rk, dh64 = up(j.rstd_out)[:, None], up(dh)
            xn, a, am = o64 * rk, dh64 * (offset + gn), dh64.abs() * (offset + gn.abs())
            d = d + rk * (a - xn * (a * xn).mean(1, keepdim=True))
            dm = dm + rk * (am + xn.abs() * (am * xn.abs()).mean(1, keepdim=True))
            within(b.dgamma_next, (dh64 * xn).sum(0), (T + 4) * U * (dh64 * xn).abs().sum(0), torch.float32, "dgn")
        else:
            assert b.dgamma_next is None
        dslack = (H + 10) * U * dm
        within(b.dx, d, dslack, dtype, "dx")
        rk = up(j.rstd_y)[:, None]
        yn, gp, gpm = y64 * rk, offset + ga, offset + ga.abs()
        gv = 1.0 if gt is None else gt
        v, vm = scale * d * gv, (scale * dm * gv).abs()
        bb, bm = v * gp, vm * gpm
        within(b.dgamma, (v * yn).sum(0), (T + H + 16) * U * (vm * yn.abs()).sum(0), torch.float32, "dgamma")
        within(b.dy, rk * (bb - yn * (bb * yn).mean(1, keepdim=True)),
               (2 * H + 24) * U * rk * (bm + yn.abs() * (bm * yn.abs()).mean(1, keepdim=True)), dtype, "dy")
        dg, dgm = scale * d * yn * gp, abs(scale) * dm * yn.abs() * gpm
        if kind == "none":
            assert b.dgate is None
        elif kind == "full":
            within(b.dgate, dg, (H + 16) * U * dgm, dtype, "dgate")
        elif kind == "channel":
            within(b.dgate, dg.sum(0), (T + H + 16) * U * dgm.sum(0), torch.float32, "dgate")
        else:
            within(b.dgate, dg.sum(1, keepdim=True), (2 * H + 16) * U * dgm.sum(1, keepdim=True), torch.float32,
                   "dgate")


def test_join_in_place(M):
    """out may be x: the C call on the same buffer gives the same bits."""
    from routing_grouped_gemm_router_gb300 import _lib as L
    g, T, H = gen(5), 50, 1000
    x, y, gamma = randn(g, T, H, dtype=torch.bfloat16), randn(g, T, H, dtype=torch.bfloat16), randn(g, H)
    j = M.block_join(x, y, gamma)
    r = torch.empty(T, device=DEV)
    L.moe_block_join(L.moe_block_t(T, H, L.MOE_BF16, 0, 1.0, 0.0, 1e-6), x, y, gamma, None, None, x, r, None, None)
    assert torch.equal(x, j.out) and torch.equal(r, j.rstd_y)


# ----------------------------------------------------------------------------------- router
def route64(z, ids, mode, renorm, scale):
    """The router weights of the chosen ids in 64 bits (differentiable)."""
    if mode == 0:
        p = torch.softmax(z.gather(1, ids), 1) if renorm else torch.softmax(z, 1).gather(1, ids)
        return scale * p
    s = torch.sigmoid(z.gather(1, ids))
    return scale * (s / s.sum(1, keepdim=True) if renorm else s)


@pytest.mark.parametrize("mode,renorm", [(0, True), (0, False), (1, True), (1, False)])
@pytest.mark.parametrize("T,E,k,ns", [(1, 1, 1, 0), (5, 8, 2, 0), (9, 128, 8, 1), (300, 256, 8, 0), (17, 500, 32, 0),
                                      (3, 37, 5, 2)])
def test_route_backward(M, L, T, E, k, ns, mode, renorm):
    g = gen(T + E)
    logits, bias = randn(g, T, E, std=3.0), randn(g, E) if mode == 0 else None
    cfg = L.make_config(T, 8, 8, E, k, L.MOE_F32, mode, renorm, 2.5, n_group=1, topk_group=1, logit_bias=bias,
                        n_shared=ns)
    assert cfg.k == k
    z = (logits + bias if mode == 0 else logits).to(F64).requires_grad_()
    ids = z.detach().topk(k, dim=1).indices
    slots = torch.full((T, k + ns), E, dtype=torch.int32, device=DEV)
    slots[:, :k] = ids.to(torch.int32)
    dw = randn(g, T, k + ns)
    w = route64(z, ids, mode, renorm, 2.5)
    (w * dw[:, :k].to(F64)).sum().backward()
    got = M.route_backward(logits, slots, dw, mode=mode, renormalize=renorm, scale=2.5, logit_bias=bias, n_shared=ns)
    # p and s: expf of an argument below 64 in magnitude that is off by a few units (64 * 2^-24 * 3
    # relative), sums of up to E terms, the divide; then a difference of terms of this magnitude
    amp = dw[:, :k].abs().to(F64).max(1, keepdim=True).values
    rel = (E + 256) * U
    wm = torch.zeros_like(z).scatter_(1, ids, w.detach().abs())
    if mode == 0 and not renorm:
        wm = 2.5 * torch.softmax(z.detach(), 1)
    if mode == 1 and renorm:  # ds is divided by the sum of the scores, then times s (1 - s)
        wm = wm * 2
    within(got, z.grad, rel * 4 * amp * wm, torch.float32, "dlogits")
    if not (mode == 0 and not renorm):
        assert (got == 0).sum() >= T * (E - k)

    # and against differences of the 64-bit weights along a random direction
    v = randn(g, T, E).to(F64)
    f = lambda s: (route64(z.detach() + s * v, ids, mode, renorm, 2.5) * dw[:, :k].to(F64)).sum()  # noqa: E731
    eps = 1e-5
    diff = (f(eps) - f(-eps)) / (2 * eps)
    along = (got.to(F64) * v).sum()
    # second-order error of the difference, and the kernel's bound along v
    assert (along - diff).abs() <= 1e-6 * amp.sum() + (rel * 4 * amp * wm * v.abs()).sum() + 1e-9


def test_route_backward_skips_ids_outside_the_range(M):
    logits = torch.zeros(2, 8, device=DEV)
    ids = torch.tensor([[0, -1], [9, 3]], dtype=torch.int32, device=DEV)
    got = M.route_backward(logits, ids, torch.ones(2, 2, device=DEV), mode=1, renormalize=False)
    want = torch.zeros(2, 8, device=DEV)
    want[0, 0] = want[1, 3] = 0.25
    assert torch.equal(got, want)


# ----------------------------------------------------------- gradients against differences
def test_join_gradient_against_differences(M):
    """Directional differences of the 64-bit join against the kernels' gradients (fp32)."""
    g, T, H, eps = gen(11), 6, 264, 1e-5
    names = ["x", "y", "gamma", "gate", "gamma_next"]
    v = dict(x=randn(g, T, H), y=randn(g, T, H), gamma=1 + randn(g, H, std=0.2),
             gate=torch.sigmoid(randn(g, H)), gamma_next=1 + randn(g, H, std=0.2))
    dres, dh = randn(g, T, H), randn(g, T, H)
    j = M.block_join(v["x"], v["y"], v["gamma"], gate=v["gate"], scale=0.5, gamma_next=v["gamma_next"])
    b = M.block_join_backward(dres, v["y"], v["gamma"], j.rstd_y, gate=v["gate"], scale=0.5, dh=dh, out=j.out,
                              gamma_next=v["gamma_next"], rstd_out=j.rstd_out)
    grads = dict(x=b.dx, y=b.dy, gamma=b.dgamma, gate=b.dgate, gamma_next=b.dgamma_next)

    def loss(w):
        out, _, h, _ = join64(w["x"], w["y"], w["gamma"], w["gate"], 0.5, w["gamma_next"], 1e-6, 0.0, torch.float32)
        return (out * dres.to(F64)).sum() + (h * dh.to(F64)).sum()
    base = {n: t.to(F64) for n, t in v.items()}
    for n in names:
        u = randn(g, *v[n].shape).to(F64)
        at = lambda s: loss({**base, n: base[n] + s * u})  # noqa: E731
        diff = (at(eps) - at(-eps)) / (2 * eps)
        along = (grads[n].to(F64) * u).sum()
        # a difference's own error is of order eps^2 times third derivatives; fp32 adds ~(T + H) units a term
        tol = 1e-6 * T * H + 2 * (T + H) * U * (grads[n].to(F64).abs() * u.abs()).sum()
        assert (along - diff).abs() <= tol, n


def test_expert_gradient_against_differences(M):
    """Directional differences of the 64-bit expert layer against the fp32 kernels' gradients."""
    H, I = 72, 40
    counts, rs, live, xs, dys, W13, W2, cnt = expert_inputs("edges", H, I, torch.float32, 21)
    h13, _ = M.expert_up(xs, W13, cnt)
    dh13, act = M.expert_down_backward(dys, W2, h13, cnt)
    grads = {"xs": M.expert_up_backward(dh13, W13, cnt), "W13": M.expert_weight_grad(dh13, xs, cnt),
             "W2": M.expert_weight_grad(dys, act, cnt)}
    base = {"xs": xs.to(F64), "W13": W13.to(F64), "W2": W2.to(F64)}

    def loss(w):
        s = 0.0
        for e, r in rs:
            h = w["xs"][r] @ w["W13"][e].T
            s = s + (((torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ w["W2"][e].T) * dys[r].to(F64)).sum()
        return s
    g, eps = gen(22), 1e-5
    for n, t in base.items():
        u = randn(g, *t.shape).to(F64) * (live if n == "xs" else 1)
        at = lambda s: loss({**base, n: t + s * u})  # noqa: E731
        diff = (at(eps) - at(-eps)) / (2 * eps)
        along = (grads[n].to(F64) * u).sum()
        tol = 1e-6 * sum(counts) * H + 600 * U * (grads[n].to(F64).abs() * u.abs()).sum()
        assert (along - diff).abs() <= tol, n


# ------------------------------------------------------------------- streams, graphs, bits
def whole_pass(M, x, ids, topk_w, W13, W2, gamma, dout, E):
    h, r = M.block_norm(x, gamma)
    t = M.sort_tokens(ids, E)
    xs, pos = M.permute(h, ids, t.sorted_ids, E)
    h13, act = M.expert_up(xs, W13, t.counts)
    ys = M.expert_down(act, W2, t.counts)
    y = M.unpermute(ys, pos, topk_w)
    j = M.block_join(x, y, gamma, scale=0.5)
    b = M.block_join_backward(dout, y, gamma, j.rstd_y, scale=0.5)
    dys, dw = M.unpermute_backward(b.dy, ys, t.sorted_ids, pos, topk_w)
    dh13, act = M.expert_down_backward(dys, W2, h13, t.counts)
    dxs = M.expert_up_backward(dh13, W13, t.counts)
    dW13, dW2 = M.expert_weight_grad(dh13, xs, t.counts), M.expert_weight_grad(dys, act, t.counts)
    dx, dg = M.block_norm_backward(M.permute_backward(dxs, pos), x, gamma, r, dres=b.dx)
    return [j.out, dx, dg, b.dgamma, dw, dW13, dW2]


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_step_on_another_stream_and_in_a_graph(M, dtype):
    """The same bits from run to run, on a side stream, and from a captured graph that is replayed
    on new inputs."""
    T, k, E, H, I = 150, 3, 10, 264, 136
    g = gen(2)
    def inputs(seed):
        s = gen(seed)
        return [randn(s, T, H, dtype=dtype), random_ids(s, T, k, E, None),
                torch.softmax(randn(s, T, k), 1), randn(s, T, H, dtype=dtype)]
    W13, W2 = randn(g, E, 2 * I, H, dtype=dtype, std=0.1), randn(g, E, H, I, dtype=dtype, std=0.1)
    gamma = 1 + randn(g, H, std=0.1)
    x, ids, w, dout = inputs(5)
    ref = whole_pass(M, x, ids, w, W13, W2, gamma, dout, E)
    again = whole_pass(M, x, ids, w, W13, W2, gamma, dout, E)
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = whole_pass(M, x, ids, w, W13, W2, gamma, dout, E)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = whole_pass(M, x, ids, w, W13, W2, gamma, dout, E)
    for seed in (5, 6):
        new = inputs(seed)
        want = whole_pass(M, new[0], new[1], new[2], W13, W2, gamma, new[3], E)
        for a, b in zip((x, ids, w, dout), new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_a_buffer_past_two_to_the_31_elements(M):
    """Rows whose element offsets pass 32 bits."""
    T, k, E, H = 20000, 8, 16, 16384  # 160,240 rows: 2.6 G elements of bf16
    g = gen(4)
    ids = torch.rand(T, E, generator=g, device=DEV).topk(k, dim=1).indices.to(torch.int32)
    x = randn(g, T, H, dtype=torch.bfloat16)
    t = M.sort_tokens(ids, E)
    xs, pos = M.permute(x, ids, t.sorted_ids, E)
    assert xs.numel() > 1 << 31
    assert int(pos.max()) * H > 1 << 31
    last = pos.argmax()
    assert torch.equal(xs[pos.view(-1)[last].long()], x[last // k])
    w = torch.full((T, k), 0.125, device=DEV)
    out = M.unpermute(xs, pos, w)  # eight equal rows an eighth each: exact
    assert torch.equal(out, x)
    dys, dw = M.unpermute_backward(x, xs, t.sorted_ids, pos, w)
    assert torch.equal(dys[pos.view(-1)[last].long()], x[last // k] * 0.125)
    want = x.to(F64).square().sum(1)
    within(dw, want[:, None].expand(T, k), (H + 2) * U * want[:, None].expand(T, k), torch.float32, "dw")
