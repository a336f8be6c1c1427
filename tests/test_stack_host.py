"""Operators around a stack's blocks, host side: what their entry points refuse, sizes, and the
wrappers' checks of tensors, all before anything is enqueued and without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import _lib
    return _lib


@pytest.fixture(scope="module")
def M(L):
    from routing_grouped_gemm_router_gb300 import training
    return training


def refused(L, status, fn, *a, **kw):
    with pytest.raises(L.MoeError) as ei:
        fn(*a, stream=0, **kw) if "size" not in fn.__name__ else fn(*a)
    assert ei.value.status == status


def test_entry_points_are_bound(L):
    import routing_grouped_gemm_router_gb300 as pkg
    names = [n for n in L.EXPORTED if n.startswith(("moe_embed", "moe_layer", "moe_dropout", "moe_balance"))]
    assert len(names) == 12
    for n in names:
        assert callable(getattr(L, n)) and getattr(pkg, n) is getattr(L, n)
    assert ctypes.sizeof(L.moe_layer_t) == 20 and ctypes.sizeof(L.moe_drop_t) == 24
    assert ctypes.sizeof(L.moe_balance_t) == 56


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(H=0), 1), (dict(H=12), 1), (dict(T=(1 << 28) + 1), 2),
    (dict(V=(1 << 26) + 1), 2), (dict(H=(1 << 20) + 8), 2), (dict(tb=2), 1), (dict(dtype=2), 1), (dict(tok=0), 1),
    (dict(tok=20, tb=8), 1), (dict(rows=24), 1), (dict(out=0), 1), (dict(out=8), 1)])
def test_embed_refuses(L, kw, status):
    a = dict(T=4, V=10, H=64, tb=4, dtype=L.MOE_BF16, tok=16, rows=16, out=16) | kw
    refused(L, status, L.moe_embed, a["tok"], a["tb"], a["T"], a["rows"], a["V"], a["H"], a["dtype"], 1.0, a["out"])
    refused(L, status, L.moe_embed_backward, a["rows"], a["tok"], a["tb"], a["T"], a["V"], a["H"], a["dtype"],
            L.MOE_F32, 1.0, 0, a["out"], 16, 1 << 60)
    if set(kw) <= {"T", "V", "H"}:
        refused(L, status, L.moe_embed_workspace_size, a["T"], a["V"], a["H"])


def test_embed_backward_refuses_types_and_workspaces(L):
    ws = L.moe_embed_workspace_size(100, 10, 64)
    assert ws >= 100 * 16
    args = lambda dt, out: (16, 16, 4, 100, 10, 64, dt, out, 1.0, 0, 16)  # noqa: E731
    refused(L, 1, L.moe_embed_backward, *args(L.MOE_F32, L.MOE_BF16), 16, ws)
    refused(L, 1, L.moe_embed_backward, *args(L.MOE_BF16, 5), 16, ws)
    for p, n in ((0, ws), (8, ws), (16, ws - 1)):
        refused(L, 3, L.moe_embed_backward, *args(L.MOE_BF16, L.MOE_F32), p, n)


def layer(L, T=4, H=64, dtype=1, eps=1e-5, scale=1.0):
    return L.moe_layer_t(T, H, dtype, eps, scale)


def drop(L, p=0.1, rng=16, site=0):
    return L.moe_drop_t(p, rng, site)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(H=4), 1), (dict(H=68), 1), (dict(dtype=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(H=32776), 2), (dict(T=(1 << 30) + 1), 2)])
def test_layer_calls_refuse_bad_sizes(L, kw, status):
    c, d = layer(L, **kw), drop(L)
    refused(L, status, L.moe_layer_workspace_size, c)
    refused(L, status, L.moe_layer_norm, c, 16, 16, 0, 16, 16, 16)
    refused(L, status, L.moe_layer_norm_backward, c, 16, 16, 16, 16, 16, 0, 16, 16, 0, 16, 1 << 40)
    refused(L, status, L.moe_dropout, c, d, 16, 16)
    refused(L, status, L.moe_dropout_join, c, d, 16, 16, 0, 0, 16, 0, 0, 0)
    refused(L, status, L.moe_dropout_join_backward, c, d, 0, 16, 16, 16, 16, 16, 16, 16, 16, 0, 16, 1 << 40)


@pytest.mark.parametrize("kw", [dict(p=-0.1), dict(p=1.0), dict(p=float("nan")), dict(p=1 - 2.0 ** -40),
                                dict(rng=0), dict(rng=20), dict(p=1e-30, rng=0)])
def test_dropout_calls_refuse_bad_probabilities(L, kw):
    c, d = layer(L), drop(L, **kw)
    refused(L, 1, L.moe_dropout, c, d, 16, 16)
    refused(L, 1, L.moe_dropout_join, c, d, 16, 16, 0, 0, 16, 0, 0, 0)
    refused(L, 1, L.moe_dropout_join_backward, c, d, 0, 16, 16, 16, 16, 16, 16, 16, 16, 0, 16, 1 << 40)


def test_layer_calls_refuse_bad_pointers(L):
    c, d = layer(L), drop(L)
    ws = L.moe_layer_workspace_size(c)
    assert ws >= 2 * 64 * 4
    ok = [16, 16, 16, 16, 16, 16]  # x, gamma, beta, h, mean, rstd
    for at, p in ((0, 0), (0, 8), (1, 0), (1, 8), (2, 8), (3, 0), (3, 24), (4, 0), (5, 2)):
        refused(L, 1, L.moe_layer_norm, c, *(ok[:at] + [p] + ok[at + 1:]))
    ok = [16] * 9  # dh, x, gamma, mean, rstd, dres, dx, dgamma, dbeta
    for at, p in ((0, 8), (1, 0), (2, 0), (3, 0), (4, 1), (5, 8), (6, 0), (7, 0), (8, 2)):
        refused(L, 1, L.moe_layer_norm_backward, c, *(ok[:at] + [p] + ok[at + 1:]), 16, ws)
    for p, n in ((0, ws), (8, ws), (16, ws - 1)):
        refused(L, 3, L.moe_layer_norm_backward, c, *ok, p, n)
        refused(L, 3, L.moe_dropout_join_backward, c, d, *[16] * 10, p, n)
    refused(L, 1, L.moe_dropout, c, d, 8, 16)
    refused(L, 1, L.moe_dropout, c, d, 16, 0)
    # a next norm's arguments come together
    for at in range(2, 7):
        p = [16, 16, 0, 0, 16, 0, 0, 0]
        p[at if at < 4 else at + 1] = 16
        refused(L, 1, L.moe_dropout_join, c, d, *p)
    for at in range(10):  # dres, dh, out, gamma_next, mean, rstd, dx, dy, dgamma_next, dbeta_next
        p = [16] * 10
        p[at] = 2 if at in (0, 9) else 0
        refused(L, 1, L.moe_dropout_join_backward, c, d, *p, 16, ws)


def balance(L, T=10, E=8, k=2, n_shared=0, mode=0, bias=0, S=1, offsets=0, mask=0):
    return L.moe_balance_t(T, E, k, n_shared, mode, bias, S, offsets, mask)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(k=33, E=64), 1), (dict(n_shared=-1), 1),
    (dict(n_shared=31), 1), (dict(mode=2), 1), (dict(S=0, offsets=16), 1), (dict(S=2), 1), (dict(bias=2), 1),
    (dict(offsets=18), 1), (dict(E=513), 2), (dict(T=(1 << 28) + 1), 2), (dict(S=(1 << 20) + 1, offsets=16), 2)])
def test_balance_refuses(L, kw, status):
    c = balance(L, **kw)
    refused(L, status, L.moe_balance_workspace_size, c)
    refused(L, status, L.moe_balance_loss, c, *[16] * 7, 16, 1 << 60)
    refused(L, status, L.moe_balance_loss_backward, c, 16, 16, 16, 16, 16, 0, 16)


def test_balance_refuses_bad_pointers(L):
    c = balance(L)
    ws = L.moe_balance_workspace_size(c)
    for at in range(7):
        p = [16] * 7
        p[at] = 0
        refused(L, 1, L.moe_balance_loss, c, *p, 16, ws)
    for p, n in ((0, ws), (8, ws), (16, ws - 1)):
        refused(L, 3, L.moe_balance_loss, c, *[16] * 7, p, n)
    for at in range(6):
        p = [16] * 6
        p[at] = 0
        refused(L, 1, L.moe_balance_loss_backward, c, *p[:5], 0, p[5])


def test_wrappers_refuse_tensors_that_do_not_fit(M):
    f, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    x, tok, g = torch.zeros(4, 64, dtype=bf), torch.zeros(4, dtype=i32), torch.zeros(64)
    logits, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=i32)
    cases = [
        (lambda: M.embed(tok, x), "table: has to be on a CUDA"),
        (lambda: M.embed(tok, x.half()), "table: dtype"),
        (lambda: M.embed_backward(x[:, ::2], tok, 9), "dx: has to be contiguous"),
        (lambda: M.layer_norm(x[0], g), "x: shape"),
        (lambda: M.layer_norm_backward(x, x.double(), g, g, g), "x: dtype"),
        (lambda: M.dropout(x.long(), 0.1), "x: dtype"),
        (lambda: M.dropout_join(x.t(), x, 0.1), "x: has to be contiguous"),
        (lambda: M.dropout_join_backward(None), "dres or dh: a gradient"),
        (lambda: M.dropout_join_backward(x, dh=x, out=x), "dh, out, gamma_next, mean and rstd are given together"),
        (lambda: M.dropout_join_backward(x, mean=g), "dh, out, gamma_next, mean and rstd are given together"),
        (lambda: M.balance_loss(logits.to(bf), ids), "logits: dtype"),
        (lambda: M.balance_loss(logits[0], ids), "logits: shape"),
    ]
    for fn, said in cases:
        with pytest.raises(ValueError, match=said):
            fn()


def calls_on(M, dev):
    """A call of every operator whose tensors, none of which has memory, lie on `dev`."""
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
    f, i32 = torch.float32, torch.int32
    x, tok, g, r, rng = t(4, 64), t(4, dtype=i32), t(64, dtype=f), t(4, dtype=f), t(2, dtype=torch.int64)
    logits, ids, two = t(4, 8, dtype=f), t(4, 2, dtype=i32), t(2, dtype=f)
    saved = M.BalanceLoss(two, t(1, 8, dtype=i32), t(1, dtype=i32), t(1, 8, dtype=f), t(2, dtype=i32))
    return {
        "table": lambda: M.embed(tok, x), "dx": lambda: M.embed_backward(x, tok, 9), "x": lambda: M.layer_norm(x, g),
        "x ": lambda: M.layer_norm_backward(x, x, g, r, r), "x  ": lambda: M.dropout(x, 0.1, rng),
        "x   ": lambda: M.dropout_join(x, x, 0.1, rng),
        "out": lambda: M.dropout_join_backward(x, 0.1, rng, dh=x, out=x, gamma_next=g, mean=r, rstd=r),
        "logits": lambda: M.balance_loss(logits, ids),
        "logits ": lambda: M.balance_loss_backward(two, logits, saved, 2)}


def test_wrappers_refuse_tensors_of_a_device_that_is_not_current(M, monkeypatch):
    """Kernels start on the calling thread's device, whatever device a tensor's addresses belong to."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    from routing_grouped_gemm_router_gb300 import _native_stack
    with monkeypatch.context() as m, FakeTensorMode():
        m.setattr(torch.cuda, "is_available", lambda: False)  # no second GPU is touched to describe it
        calls = calls_on(M, "cuda:1")
    assert len(calls) == len([n for n in dir(_native_stack) if not n.startswith("__") and n != "set_error"])
    for name, fn in calls.items():
        with pytest.raises(ValueError, match=f"^{name.strip()}: is on cuda:1, which is not the current device"):
            fn()
