"""Training operators, host side: what their entry points refuse, sizes, and the wrappers'
checks of tensors, all before anything is enqueued and without a GPU."""
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
        fn(*a, **kw)
    assert ei.value.status == status


def test_entry_points_are_bound(L):
    for n in ("moe_permute", "moe_unpermute_backward", "moe_expert_weight_grad", "moe_block_join_backward",
              "moe_route_backward"):
        assert n in L.EXPORTED and callable(getattr(L, n))


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(k=0), 1), (dict(k=33), 1), (dict(H=12), 1), (dict(H=0), 1), (dict(rows=0), 1),
    (dict(dtype=2), 1), (dict(T=1 << 26, k=32), 2), (dict(rows=(1 << 28) + 16), 2)])
def test_dispatch_refuses_bad_sizes(L, kw, status):
    a = dict(T=4, k=2, H=64, dtype=L.MOE_BF16, rows=64)
    a.update(kw)
    T, k, H, dt, rows = a["T"], a["k"], a["H"], a["dtype"], a["rows"]
    refused(L, status, L.moe_permute, 16, 16, 16, T, k, 8, H, dt, rows, 16, 16, stream=0)
    refused(L, status, L.moe_permute_backward, 16, 16, T, k, H, dt, rows, 16, stream=0)
    refused(L, status, L.moe_unpermute, 16, 16, 16, T, k, H, dt, rows, 16, stream=0)
    refused(L, status, L.moe_unpermute_backward, 16, 16, 16, 16, 16, T, k, H, dt, rows, 16, 16, stream=0)


def test_dispatch_refuses_bad_pointers(L):
    tail = (4, 2, 64, L.MOE_BF16, 64)
    refused(L, 1, L.moe_permute, 16, 16, 16, 4, 2, 0, 64, L.MOE_BF16, 64, 16, 16, stream=0)  # no expert
    for bad in range(5):  # null, then rows off a 16-byte boundary
        p = [16] * 5
        p[bad] = 0
        refused(L, 1, L.moe_permute, p[0], p[1], p[2], 4, 2, 8, 64, L.MOE_BF16, 64, p[3], p[4], stream=0)
    refused(L, 1, L.moe_permute, 24, 16, 16, 4, 2, 8, 64, L.MOE_BF16, 64, 16, 16, stream=0)
    refused(L, 1, L.moe_permute_backward, 16, 18, *tail, 16, stream=0)
    refused(L, 1, L.moe_unpermute, 16, 16, 0, *tail, 16, stream=0)
    refused(L, 1, L.moe_unpermute, 16, 16, 16, *tail, 8, stream=0)
    refused(L, 1, L.moe_unpermute_backward, 16, 16, 16, 16, 16, *tail, 16, 0, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 1), (dict(E=0), 1), (dict(H=20), 1), (dict(I=4), 1), (dict(dtype=7), 1), (dict(E=513), 2),
    (dict(H=(1 << 20) + 8), 2)])
def test_experts_refuse_bad_sizes(L, kw, status):
    a = dict(rows=64, E=4, H=64, I=96, dtype=L.MOE_BF16)
    a.update(kw)
    c = L.moe_experts_t(a["rows"], a["E"], a["H"], a["I"], a["dtype"])
    refused(L, status, L.moe_expert_up, c, 16, 16, 16, 16, 16, stream=0)
    refused(L, status, L.moe_expert_down, c, 16, 16, 16, 16, stream=0)
    refused(L, status, L.moe_expert_down_backward, c, 16, 16, 16, 16, 16, 16, stream=0)
    refused(L, status, L.moe_expert_up_backward, c, 16, 16, 16, 16, stream=0)


def test_experts_refuse_bad_pointers(L):
    c = L.moe_experts_t(64, 4, 64, 96, L.MOE_BF16)
    refused(L, 1, L.moe_expert_up, c, 16, 16, 0, 16, 16, stream=0)
    refused(L, 1, L.moe_expert_down, c, 16, 16, 16, 8, stream=0)
    refused(L, 1, L.moe_expert_down_backward, c, 16, 16, 0, 16, 16, 16, stream=0)
    refused(L, 1, L.moe_expert_up_backward, c, 16, 0, 16, 16, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), 1), (dict(E=0), 1), (dict(M=12), 1), (dict(N=0), 1), (dict(dt=0, odt=1), 1), (dict(odt=2), 1),
    (dict(E=600), 2), (dict(dW=0), 1), (dict(dW=8), 1), (dict(counts=0), 1)])
def test_weight_grad_refuses(L, kw, status):
    a = dict(rows=64, E=4, M=64, N=96, dt=1, odt=0, dW=16, counts=16)
    a.update(kw)
    refused(L, status, L.moe_expert_weight_grad, a["rows"], a["E"], a["M"], a["N"], a["dt"], a["odt"], 0, 16, 16,
            a["counts"], a["dW"], stream=0)


def block(L, T=4, H=64, dtype=1, gate=0, scale=1.0, offset=0.0, eps=1e-6):
    return L.moe_block_t(T, H, dtype, gate, scale, offset, eps)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(H=4), 1), (dict(H=68), 1), (dict(dtype=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(H=32776), 2)])
def test_block_calls_refuse_bad_sizes(L, kw, status):
    c = block(L, **kw)
    refused(L, status, L.moe_block_workspace_size, c)
    refused(L, status, L.moe_block_norm, c, 16, 16, 16, 16, stream=0)
    refused(L, status, L.moe_block_norm_backward, c, 16, 16, 16, 16, 0, 16, 16, 16, 1 << 40, stream=0)
    refused(L, status, L.moe_block_join, c, 16, 16, 16, 0, 0, 16, 16, 0, 0, stream=0)
    refused(L, status, L.moe_block_join_backward, c, 16, 0, 0, 16, 16, 0, 0, 16, 0, 16, 16, 16, 0, 0, 16, 1 << 40,
            stream=0)


def test_block_calls_refuse_bad_pointers(L):
    c, g = block(L), block(L, gate=L.MOE_GATE_CHANNEL)
    ws = L.moe_block_workspace_size(c)
    assert ws >= 64 * 4
    refused(L, 1, L.moe_block_norm, c, 16, 0, 16, 16, stream=0)
    refused(L, 1, L.moe_block_norm, c, 16, 16, 16, 0, stream=0)
    refused(L, 1, L.moe_block_norm_backward, c, 16, 16, 16, 16, 8, 16, 16, 16, ws, stream=0)
    refused(L, 3, L.moe_block_norm_backward, c, 16, 16, 16, 16, 0, 16, 16, 0, ws, stream=0)
    refused(L, 3, L.moe_block_norm_backward, c, 16, 16, 16, 16, 0, 16, 16, 16, ws - 1, stream=0)
    # a gate without its kind, a kind without its gate, a kind that does not exist
    refused(L, 1, L.moe_block_join, c, 16, 16, 16, 16, 0, 16, 16, 0, 0, stream=0)
    refused(L, 1, L.moe_block_join, g, 16, 16, 16, 0, 0, 16, 16, 0, 0, stream=0)
    refused(L, 1, L.moe_block_join, block(L, gate=4), 16, 16, 16, 16, 0, 16, 16, 0, 0, stream=0)
    # half a next norm
    refused(L, 1, L.moe_block_join, c, 16, 16, 16, 0, 16, 16, 16, 0, 16, stream=0)
    refused(L, 1, L.moe_block_join, c, 16, 16, 16, 0, 0, 16, 16, 16, 16, stream=0)

    def back(cfg=c, dres=16, dh=0, out=0, gate=0, gn=0, ro=0, dgn=0, dgate=0, w=ws):
        return L.moe_block_join_backward(cfg, dres, dh, out, 16, 16, gate, gn, 16, ro, 16, 16, 16, dgn, dgate, 16, w,
                                         stream=0)
    refused(L, 1, back, dres=0)                                   # no gradient at all
    refused(L, 1, back, dh=16, out=16, gn=16, ro=16)              # next norm without its gradient's place
    refused(L, 1, back, cfg=g, gate=16)                           # gate without its gradient's place
    refused(L, 1, back, dgate=16)
    refused(L, 3, back, w=ws - 1)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(mode=2), 1), (dict(n_shared=9), 1), (dict(E=520), 2)])
def test_route_backward_refuses(L, kw, status):
    a = dict(T=4, E=8, k=2, mode=0, n_shared=0)
    a.update(kw)
    c = L.make_config(a["T"], 8, 8, a["E"], a["k"], L.MOE_F32, a["mode"], n_shared=a["n_shared"])
    refused(L, status, L.moe_route_backward, c, 16, 16, 16, 16, stream=0)
    if not kw.get("E"):
        refused(L, 1, L.moe_route_backward, L.make_config(4, 8, 8, 8, 2, L.MOE_F32), 16, 16, 16, 0, stream=0)


def test_wrappers_refuse_wrong_tensors(M):
    """Shapes, types, strides and devices are refused by name before any call."""
    f, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    x, ids = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 2, dtype=i32)
    cases = [
        (lambda: M.permute(x, ids, torch.zeros(64, dtype=i32), 8), "x: has to be on a CUDA"),
        (lambda: M.permute(x.half(), ids, torch.zeros(64, dtype=i32), 8), "x: dtype"),
        (lambda: M.permute(x[:, ::2], ids, torch.zeros(64, dtype=i32), 8), "x: has to be contiguous"),
        (lambda: M.sort_tokens(ids.long(), 8), "topk_ids: dtype"),
        (lambda: M.sort_tokens(ids.reshape(-1), 8), "topk_ids: shape"),
        (lambda: M.expert_weight_grad(x[0], x, ids), "dy: shape"),
        (lambda: M.block_norm(x.reshape(2, 2, 64), torch.zeros(64)), "x: shape"),
        (lambda: M.route_backward(x, ids, torch.zeros(4, 2)), "logits: dtype"),
    ]
    for fn, said in cases:
        with pytest.raises(ValueError, match=said):
            fn()


def calls_on(M, dev):
    """A call of every operator whose tensors, none of which has memory, lie on `dev`."""
    f, bf, i32 = torch.float32, torch.bfloat16, torch.int32
    t = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype, device=dev)  # noqa: E731
    T, k, E, H, I, P = 4, 2, 8, 64, 48, 128
    x, ids, w = t(T, H), t(T, k, dtype=i32), t(T, k, dtype=f)
    rows, sid, cnt = t(P, H), t(P, dtype=i32), t(E, dtype=i32)
    W13, W2, act, h13, dh13 = t(E, 2 * I, H), t(E, H, I), t(P, I), t(P, 2 * I, dtype=f), t(P, 2 * I)
    g, r, logits = t(H, dtype=f), t(T, dtype=f), t(T, E, dtype=f)
    return {
        "topk_ids": lambda: M.sort_tokens(ids, E), "x": lambda: M.permute(x, ids, sid, E),
        "dxs": lambda: M.permute_backward(rows, ids), "ys": lambda: M.unpermute(rows, ids, w),
        "ys ": lambda: M.unpermute_backward(x, rows, sid, ids, w), "xs": lambda: M.expert_up(rows, W13, cnt),
        "act": lambda: M.expert_down(act, W2, cnt), "dys": lambda: M.expert_down_backward(rows, W2, h13, cnt),
        "dh13": lambda: M.expert_up_backward(dh13, W13, cnt), "dy": lambda: M.expert_weight_grad(rows, act, cnt),
        "x ": lambda: M.block_norm(x, g), "x  ": lambda: M.block_norm_backward(x, x, g, r),
        "x   ": lambda: M.block_join(x, x, g), "y": lambda: M.block_join_backward(x, x, g, r),
        "logits": lambda: M.route_backward(logits, ids, w)}


def test_wrappers_refuse_tensors_of_a_device_that_is_not_current(M, monkeypatch):
    """Kernels start on the calling thread's device, whatever device a tensor's addresses belong to."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    from routing_grouped_gemm_router_gb300 import _native
    with monkeypatch.context() as m, FakeTensorMode():
        m.setattr(torch.cuda, "is_available", lambda: False)  # no second GPU is touched to describe it
        calls = calls_on(M, "cuda:1")
    assert len(calls) == len([n for n in dir(_native) if not n.startswith("__") and n != "set_error"])
    for name, fn in calls.items():
        with pytest.raises(ValueError, match=f"^{name.strip()}: is on cuda:1, which is not the current device"):
            fn()


def test_buffer_rows(M):
    assert M.buffer_rows(1, 1, 1) == 16
    assert M.buffer_rows(4096, 8, 256) == (4096 * 8 + 256 * 15) // 16 * 16
    assert M.buffer_rows(3, 2, 512) == 6 * 16


def test_block_refuses_parameters_that_do_not_fit(M):
    from routing_grouped_gemm_router_gb300.sparse_block import SparseBlock, SparseStack
    g = torch.ones(64)
    ok = dict(Wg=torch.zeros(4, 64), W13=torch.zeros(4, 96, 64), W2=torch.zeros(4, 64, 48))
    SparseBlock(**ok, gamma_in=g, gamma_out=g, k=2)
    for kw in (dict(W13=torch.zeros(5, 96, 64)), dict(W2=torch.zeros(4, 64, 40)), dict(W2=torch.zeros(4, 72, 48)),
               dict(W13=torch.zeros(4, 96, 72))):
        with pytest.raises(ValueError):
            SparseBlock(**{**ok, **kw}, gamma_in=g, gamma_out=g, k=2)
    with pytest.raises(ValueError):
        SparseStack([])
