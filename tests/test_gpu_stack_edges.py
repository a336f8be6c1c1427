"""The operators around a stack's blocks at the edges of what their documentation allows: many
sequences, views that start off a 16-byte boundary, long runs of one token, values that are not
finite, calls side by side, and what the wrappers refuse on a GPU. Tolerances as in test_gpu_stack."""
import numpy as np
import pytest
import torch

from test_gpu_stack import BF, DEV, F32, F64, U, balance_ref, gen, norm_ref, randn, sums, within

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("S,E,mode", [(2047, 8, 0), (2048, 24, 1), (5000, 6, 0)])
def test_balance_of_many_sequences(M, L, S, E, mode):
    """Around the number of offsets that fit shared memory; most sequences hold a token or none."""
    g = gen(S)
    T, k = 2500, 2
    logits = randn(g, T, E)
    ids = logits.topk(k, 1).indices.to(torch.int32)
    offsets = torch.randint(3, T - 2, (S + 1,), generator=g, device=DEV).sort().values.to(torch.int32)
    up = torch.tensor([0.5, 0.1], device=DEV)
    ref = balance_ref(logits, ids, mode, None, k, offsets, None, up)
    b = M.balance_loss(logits, ids, mode=mode, offsets=offsets)
    assert torch.equal(b.counts.long(), ref["counts"]) and torch.equal(b.tokens.long(), ref["n"])
    assert b.totals.tolist() == [ref["some"], int(ref["n"].sum())]
    within(b.losses, ref["losses"], ref["loss_slack"], "losses")
    within(b.prob, ref["prob"], ref["prob_slack"], "prob")
    within(M.balance_loss_backward(up, logits, b, k, mode=mode, offsets=offsets), ref["d"], ref["off"], "dlogits")
    assert L.moe_device_status(True) == 0


@pytest.mark.parametrize("E", [8, 128, 300])
def test_balance_of_logits_off_a_16_byte_boundary(M, E):
    g = gen(E)
    T, k = 333, 3
    logits = randn(g, T * E + 1)[1:].view(T, E)
    bias = randn(g, E + 3)[3:]
    assert logits.data_ptr() % 16 and logits.is_contiguous()
    ids = logits.topk(k, 1).indices.to(torch.int32)
    up = torch.tensor([0.5, 0.1], device=DEV)
    ref = balance_ref(logits, ids, 0, bias, k, None, None, up)
    b = M.balance_loss(logits, ids, logit_bias=bias)
    out = torch.zeros(T * E + 1, device=DEV)[1:].view(T, E)
    d = M.balance_loss_backward(up, logits, b, k, logit_bias=bias, dlogits=out)
    within(b.losses, ref["losses"], ref["loss_slack"], "losses")
    within(d, ref["d"], ref["off"] + U * ref["d"].abs(), "dlogits")


@pytest.mark.parametrize("T,V,H,dtype", [
    (3000, 20000, 1032, F32),    # one CTA sorts behind the zeros
    (2049, 40, 264, BF), (65536, 70, 8, BF), (65537, 70, 8, BF),  # the sorts' borders
    (20011, 3, 136, F32), (140001, 2, 16, BF)])                   # runs of thousands of rows
def test_embed_backward_at_its_kernels_borders(M, T, V, H, dtype):
    g = gen(T)
    tok = torch.randint(-1, V, (T,), generator=g, device=DEV)
    dx = randn(g, T, H, dtype=dtype)
    ref, mag, n = sums(dx, tok, V)
    got = M.embed_backward(dx, tok, V, out_dtype=F32)
    within(got, ref, (n + 3) * U * mag, "dtable")
    assert torch.equal(got, M.embed_backward(dx, tok, V, out_dtype=F32))


def test_embedding_passes_values_that_are_not_finite(M):
    """Infinities and NaN reach their own id's row alone."""
    tok = torch.tensor([3, 1, 3, -1, 0], device=DEV)
    dx = torch.ones(5, 64, device=DEV)
    dx[1, 5], dx[2, 7], dx[3, 9] = float("inf"), float("nan"), float("nan")
    d = M.embed_backward(dx, tok, 5)
    want = torch.zeros(5, 64, device=DEV)
    want[0], want[1], want[3] = 1, 1, 2
    want[1, 5], want[3, 7] = float("inf"), float("nan")
    assert torch.equal(d.nan_to_num(nan=-7.0), want.nan_to_num(nan=-7.0))
    table = torch.full((5, 64), float("inf"), device=DEV)
    x = M.embed(tok, table, 2.0)
    assert (x[3] == 0).all() and torch.isinf(x[[0, 1, 2, 4]]).all()


@pytest.mark.parametrize("T,H", [(5, 264), (700, 2880)])
def test_a_row_that_is_not_finite_stays_its_own(M, T, H):
    """One bad row: every other row of the norm, the join and their gradients is as without it."""
    g = gen(T)
    x, y, dh = (randn(g, T, H, dtype=BF) for _ in range(3))
    gamma, beta, rng = 1 + randn(g, H, std=0.2), randn(g, H), torch.tensor([1, 2], device=DEV)

    def all_rows(x, dh):
        n = M.layer_norm(x, gamma, beta)
        j = M.dropout_join(x, y, 0.3, rng, gamma_next=gamma)
        good = M.layer_norm(torch.where(torch.isfinite(x), x, 0), gamma, beta)
        b = M.dropout_join_backward(dh, 0.3, rng, dh=dh, out=x, gamma_next=gamma, mean=good.mean, rstd=good.rstd)
        nb = M.layer_norm_backward(dh, x, gamma, good.mean, good.rstd, dh)
        return n.h, n.mean, n.rstd, j.out, j.h, b.dx, b.dy, nb.dx

    want = all_rows(x, dh)
    bad = T // 2
    x2, dh2 = x.clone(), dh.clone()
    x2[bad, 3], dh2[bad, 9] = float("inf"), float("nan")
    got = all_rows(x2, dh2)
    rest = torch.arange(T, device=DEV) != bad
    for a, b in zip(got, want):
        assert torch.equal(a[rest], b[rest])


def test_constant_rows_have_no_variance(M):
    """Rows of one value: the norm is its bias, whatever the value's size."""
    for H in (8, 264, 4096):
        for dtype in (BF, F32):
            x = torch.tensor([[0.0], [1.0], [-3e4], [1e-30]], device=DEV).to(dtype).expand(4, H).contiguous()
            gamma, beta = torch.full((H,), 2.0, device=DEV), torch.full((H,), 0.5, device=DEV)
            n = M.layer_norm(x, gamma, beta)
            (h, slack), (mean, dm), (r, dr) = norm_ref(x, gamma, beta, np.float32(1e-5).item())
            within(n.h, h, slack, "h")
            within(n.mean, mean, dm, "mean")
            within(n.rstd, r, dr, "rstd")


def test_two_calls_side_by_side(M):
    """The same operators on two streams at once, each with its own inputs, and again alone."""
    g = gen(12)
    sets = []
    for i in range(2):
        T, V, H, E = 3000 + i, 5000, 520, 64
        tok = torch.randint(0, V, (T,), generator=g, device=DEV)
        logits = randn(g, T, E)
        sets.append((tok, randn(g, T, H, dtype=BF), randn(g, T, H, dtype=BF), 1 + randn(g, H, std=0.1), logits,
                     logits.topk(4, 1).indices.to(torch.int32), torch.tensor([i, 7], device=DEV)))

    def run(tok, x, y, gamma, logits, ids, rng):
        j = M.dropout_join(x, y, 0.2, rng, 3, 1.0, gamma)
        b = M.dropout_join_backward(y, 0.2, rng, 3, 1.0, x, j.out, gamma, j.mean, j.rstd)
        return [j.out, j.h, b.dx, b.dy, b.dgamma_next, b.dbeta_next, M.embed_backward(b.dx, tok, 5000),
                *M.balance_loss(logits, ids)]

    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        want = run(*sets[i])
        for once in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(once, want))


def test_two_captured_graphs_share_nothing(M):
    """Two graphs of the same calls, replayed at once on two streams: workspaces are each graph's own."""
    g = gen(13)
    T, V, H = 2500, 3000, 264
    toks = [torch.randint(0, V, (T,), generator=g, device=DEV) for _ in range(2)]
    dxs = [randn(g, T, H) for _ in range(2)]
    gamma = 1 + randn(g, H, std=0.1)
    zero, one = torch.zeros(T, device=DEV), torch.ones(T, device=DEV)

    def run(i):
        n = M.layer_norm_backward(dxs[i], dxs[1 - i], gamma, zero, one)
        return [M.embed_backward(dxs[i], toks[i], V), *n]

    want = [run(i) for i in range(2)]
    graphs, held = [], []
    torch.cuda.synchronize()
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            held.append(run(i))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_what_the_wrappers_refuse(M, L):
    i32, i64 = torch.int32, torch.int64
    t = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
    x, g, rng, tok = t(4, 64), t(64, dtype=F32), t(2, dtype=i64), t(4, dtype=i32)
    r, logits, ids, two = t(4, dtype=F32), t(4, 8, dtype=F32), t(4, 2, dtype=i32), t(2, dtype=F32)
    offsets = torch.tensor([0, 2, 4], dtype=i32, device=DEV)
    b = M.balance_loss(logits, ids, offsets=offsets)
    cases = [
        (lambda: M.embed(tok.float(), x), "tokens: dtype"), (lambda: M.embed(tok.view(2, 2), x), "tokens: shape"),
        (lambda: M.embed(tok.cpu(), x), "tokens: has to be on a CUDA"),
        (lambda: M.embed_backward(x, tok[:3], 9), "tokens: shape"),
        (lambda: M.embed_backward(x, tok, 9, out=t(8, 64)), "out: shape"),
        (lambda: M.embed_backward(x, tok, 9, out=t(9, 64, dtype=torch.float16)), "out: dtype"),
        (lambda: M.embed_backward(x, tok, 9, out=t(9, 64), out_dtype=F32), "out: dtype"),
        (lambda: M.embed_backward(x, tok, 9, accumulate=True), "accumulate: needs"),
        (lambda: M.embed_backward(x, tok, 9, out_dtype=torch.float16), "out_dtype"),
        (lambda: M.embed_backward(x, tok, -1), "V: an extent"),
        (lambda: M.layer_norm(x, g.to(BF)), "gamma: dtype"), (lambda: M.layer_norm(x, g, g[:8]), "beta: shape"),
        (lambda: M.layer_norm_backward(x.float(), x, g, r, r), "dh: dtype"),
        (lambda: M.layer_norm_backward(x, x, g, r[:2], r), "mean: shape"),
        (lambda: M.layer_norm_backward(x, x, g, r, r, dres=x[:2]), "dres: shape"),
        (lambda: M.dropout(x, 0.1), "rng: .* needed"), (lambda: M.dropout(x, 1.0, rng), "p: 1.0"),
        (lambda: M.dropout(x, float("nan"), rng), "p: nan"), (lambda: M.dropout(x, 0.1, rng.int()), "rng: dtype"),
        (lambda: M.dropout(x, 0.1, t(3, dtype=i64)), "rng: shape"), (lambda: M.dropout(x, 0.1, rng, -1), "site: -1"),
        (lambda: M.dropout(x, 0.1, rng, 2 ** 32), "site: 4294967296"),
        (lambda: M.dropout(x, 0.1, rng.cpu()), "rng: has to be on a CUDA"),
        (lambda: M.dropout_join(x, x[:2], 0.0), "y: shape"),
        (lambda: M.dropout_join(x, x, 0.0, beta_next=g), "beta_next: needs gamma_next"),
        (lambda: M.dropout_join_backward(x[:2], dh=x, out=x, gamma_next=g, mean=r, rstd=r), "dres: shape"),
        (lambda: M.balance_loss(logits, ids[:2]), "topk_ids: shape"),
        (lambda: M.balance_loss(logits, ids, n_shared=2), "n_shared: 2 of 2"),
        (lambda: M.balance_loss(logits, ids, offsets=offsets[:1]), "offsets: 1 of them"),
        (lambda: M.balance_loss(logits, ids, offsets=offsets.long()), "offsets: dtype"),
        (lambda: M.balance_loss(logits, ids, mask=t(4, dtype=torch.uint8)), "mask: dtype"),
        (lambda: M.balance_loss(logits, ids, logit_bias=g), "logit_bias: shape"),
        (lambda: M.balance_loss_backward(two[:1], logits, b, 2, offsets=offsets), "dlosses: shape"),
        (lambda: M.balance_loss_backward(two, logits, b, 2), "counts: of 2 sequences, without"),
        (lambda: M.balance_loss_backward(two, logits, b, 2, offsets=offsets[:2].contiguous()), "offsets: shape"),
        (lambda: M.balance_loss_backward(two, logits, b, 2, offsets=offsets, dlogits=logits[:2]), "dlogits: shape"),
    ]
    for fn, said in cases:
        with pytest.raises(ValueError, match=f"^{said}"):
            fn()
    for fn in (lambda: M.embed(tok[:0], x), lambda: M.layer_norm(x[:0], g), lambda: M.dropout(x[:, :12].contiguous(), 0.0),
               lambda: M.balance_loss(logits, ids, mode=2), lambda: M.balance_loss_backward(two, logits, b, 9, offsets=offsets),
               lambda: M.layer_norm(x, g, eps=-1.0), lambda: M.embed_backward(x, tok, 0)):
        with pytest.raises(L.MoeError) as ei:
            fn()
        assert ei.value.status == 1
