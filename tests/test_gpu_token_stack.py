"""The stack that trains from token ids: its gradients against 64-bit autograd with the masks and the ids
that the kernels drew and chose, a step captured in a CUDA graph, the example."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64
H, I, E, V = 136, 72, 6, 50


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import token_stack
    return token_stack


def make(S, dtype, seed=0, n=2, k=2, ns=0, p=0.1, beta=True, bias=False, **kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    blocks = [S.TokenBlock(
        rnd(E, H, std=H ** -0.5).to(dtype), rnd(E + ns, 2 * I, H, std=H ** -0.5).to(dtype),
        rnd(E + ns, H, I, std=I ** -0.5).to(dtype), 1 + rnd(H, std=0.2), rnd(H, std=0.2) if beta else None, k,
        scale=0.7, n_shared=ns, **({"logit_bias": rnd(E)} if bias else {}), **kw) for _ in range(n)]
    stack = S.TokenStack(rnd(V, H, std=0.5).to(dtype), blocks, 1 + rnd(H, std=0.2), rnd(H, std=0.2) if beta else None,
                         embed_scale=2.0, p=p, seed=1234567890123)
    return stack, rnd


def tokens_of(T, seed, dtype=torch.int64):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = torch.randint(0, V, (T,), generator=g, device=DEV)
    if T > 4:
        t[3] = -1  # padding
    return t.to(dtype)


def factor(shape, p, rng, site):
    from test_gpu_stack import words
    if not p:
        return 1.0
    below = round(p * 2 ** 32)
    w = words(shape[0] * shape[1], int(rng[0]), int(rng[1]), site)
    return torch.from_numpy((w >= np.uint64(below)).reshape(shape)).to(DEV).to(F64) / (1 - below / 2 ** 32)


def reference(stack, saved, tokens, own, blocks64):
    """(h, losses) of the stack in 64 bits from the ids and masks of the forward pass."""
    T = len(tokens)
    ln = lambda v, ga, be: torch.nn.functional.layer_norm(v, (H,), ga, be, stack.eps)  # noqa: E731
    live = (tokens >= 0) & (tokens < V)
    x = own["table"][tokens.clamp(0, V - 1).long()] * live[:, None] * stack.embed_scale
    x = x * factor((T, H), stack.p, saved.rng, 0)
    bounds = [0, T] if saved.offsets is None else saved.offsets.tolist()
    mask = torch.ones(T, dtype=torch.bool, device=DEV) if saved.mask is None else saved.mask
    losses = []
    for i, (b, p, s) in enumerate(zip(stack.blocks, blocks64, saved.blocks)):
        h = ln(x, p["gamma"], p.get("beta"))
        logits = h @ p["Wg"].T
        z = logits + (b.logit_bias.to(F64) if b.logit_bias is not None else 0.0)
        ids = s.moe.topk_ids[:, :b.k].long()
        if b.mode == 0:
            w = torch.softmax(z.gather(1, ids), 1) if b.renormalize else torch.softmax(z, 1).gather(1, ids)
            prob = torch.softmax(z, 1)
        else:
            w = torch.sigmoid(z.gather(1, ids))
            w = w / w.sum(1, keepdim=True) if b.renormalize else w
            prob = torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
        terms, squares, N = [], 0.0, 0
        for a, e in zip(bounds[:-1], bounds[1:]):
            rows = torch.arange(a, e, device=DEV)[mask[a:e]]
            if len(rows):
                hits = torch.bincount(ids[rows].reshape(-1), minlength=E).to(F64)
                terms.append((hits * E / (b.k * len(rows)) * prob[rows].mean(0)).sum())
                squares = squares + (torch.logsumexp(z[rows], 1) ** 2).sum()
                N += len(rows)
        losses.append(torch.stack([sum(terms) / len(terms), squares / N]))
        w = torch.cat([b.router_scale * w, torch.ones(T, b.n_shared, dtype=F64, device=DEV)], 1)
        ids = s.moe.topk_ids.long()
        W13, W2 = p["W13"][ids], p["W2"][ids]
        hh = torch.einsum("th,tjih->tji", h, W13)
        act = torch.nn.functional.silu(hh[..., :b.I]) * hh[..., b.I:]
        y = (torch.einsum("tji,tjhi->tjh", act, W2) * w.unsqueeze(-1)).sum(1)
        x = x + b.scale * y * factor((T, H), stack.p, saved.rng, 1 + i)
    return ln(x, own["gamma_final"], own.get("beta_final")), torch.stack(losses)


CASES = [dict(), dict(ns=1, k=1, p=0.5), dict(mode=1, router_scale=2.5, p=0.0), dict(renormalize=False, bias=True, beta=False),
         dict(n=3, packed=True), dict(mode=1, packed=True, idt=torch.int32)]


@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_against_autograd(S, dtype, T, kw):
    kw = dict(kw)
    packed, idt = kw.pop("packed", False), kw.pop("idt", torch.int64)
    stack, rnd = make(S, dtype, seed=T, **kw)
    tokens, dh = tokens_of(T, T, idt), rnd(T, H).to(dtype)
    offsets = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device=DEV) if packed else None
    mask = tokens >= 0 if packed else None
    up = torch.tensor([0.3, 0.05], device=DEV)
    stack.rng[1] = 7
    h, losses, saved = stack.forward(tokens, offsets, mask)
    stack.rng[1] = 8  # the backward pass still draws the forward pass's masks
    stack.backward(dh, saved, up)
    own = {n: t.to(F64).requires_grad_() for n, t in stack.parameters().items()}
    blocks64 = [{n: t.to(F64).requires_grad_() for n, t in b.parameters().items()} for b in stack.blocks]
    ref, ref_losses = reference(stack, saved, tokens, own, blocks64)
    ((ref * dh.to(F64)).sum() + (ref_losses * up.to(F64)).sum()).backward()
    # A block is a chain of about 16 stages forward and backward (norm, router, products, sums, join), the
    # embedding, its dropout and the last norm 4 more; each is off by at most its type's half step, and
    # for fp32 by its sums of up to 2I + H = 280 terms, relative to the norm of its result. Errors pass
    # through later blocks with about the gain that values do, so the relative errors add.
    n = len(stack.blocks)
    tol = (16 * n + 4) * ((2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) + 280 * 2.0 ** -24)

    def near(got, want, what):
        # a gradient that is zero but for cancellation is held to the size of what cancels
        size = max(want.norm().item(), 1e-3 * dh.to(F64).norm().item())
        assert torch.isfinite(got).all(), what
        assert (got.to(F64) - want).norm() <= tol * size, f"{what}: {(got.to(F64) - want).norm() / size:.3g} > {tol:.3g}"

    near(h, ref.detach(), "h")
    assert ((losses.to(F64) - ref_losses.detach()).abs() <= tol * ref_losses.detach().abs()).all()
    for name, t in own.items():
        near(stack.grads[name], t.grad, name)
    for i, (g, p) in enumerate(zip(stack.block_grads, blocks64)):
        for name, t in p.items():
            near(g[name], t.grad, f"block {i} {name}")
    before = {n_: t.clone() for n_, t in stack.grads.items()}
    stack.backward(dh, saved, up)  # a second backward pass adds the same again
    for name, t in before.items():
        near(stack.grads[name], 2 * t.to(F64), f"twice {name}")


def test_a_captured_step_replays_with_new_inputs_and_masks(S):
    stack, rnd = make(S, torch.bfloat16, p=0.2)
    tokens, dh = tokens_of(64, 1), rnd(64, H).to(torch.bfloat16)
    up = torch.tensor([0.3, 0.05], device=DEV)

    def step():
        stack.zero_grad()
        h, losses, saved = stack.forward(tokens)
        stack.backward(dh, saved, up)
        return [h, losses, *stack.grads.values(), *(t for g in stack.block_grads for t in g.values())]

    eager_kept = step()  # results of an eager pass stay alive through the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    seen = []
    for i in (1, 2):
        tokens.copy_(tokens_of(64, 10 + i))
        stack.rng[1] = i
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        tokens.copy_(tokens_of(64, 10))
        graph.replay()
        seen.append(held[0].clone())
    assert not torch.equal(*seen)  # the same tokens, other masks
    assert all(torch.isfinite(t.float()).all() for t in eager_kept)


def test_the_example_runs():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_token_stack as ex
    eager = ex.train(steps=6)
    assert len(eager) == 6 and all(np.isfinite(eager))
    assert ex.train(steps=6, graph=True) == eager  # the same bits from replays
