"""The trainable stack: its gradients against 64-bit autograd and differences, its forward pass
against the inference layer, a step captured in a CUDA graph, the example."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_library
    build_library()
    from routing_grouped_gemm_router_gb300 import sparse_block
    return sparse_block


def make(S, dtype, seed=0, n=2, H=136, I=72, E=6, k=2, ns=0, **kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std  # noqa: E731
    bias = {"logit_bias": rnd(E)} if kw.pop("bias", False) else {}
    stack = S.SparseStack([S.SparseBlock(
        rnd(E, H, std=H ** -0.5).to(dtype), rnd(E + ns, 2 * I, H, std=H ** -0.5).to(dtype),
        rnd(E + ns, H, I, std=I ** -0.5).to(dtype), 1 + rnd(H, std=0.2), 1 + rnd(H, std=0.2), k,
        gate=0.5 + rnd(H, std=0.1) if i % 2 == 0 else None, scale=0.7, n_shared=ns, **bias, **kw) for i in range(n)])
    return stack, rnd


def reference(stack, saved, x64, dout64, blocks64):
    """The stack in 64 bits by autograd, with the ids that the kernels chose (the choice has no
    gradient). Returns (out, loss)."""
    rms = lambda v, eps: v * (v * v).mean(1, keepdim=True).add(eps).rsqrt()  # noqa: E731
    x = x64
    for b, p, s in zip(stack.blocks, blocks64, saved.blocks):
        h = rms(x, b.eps) * p["gamma_in"]
        z = h @ p["Wg"].T + (b.logit_bias.to(F64) if b.logit_bias is not None else 0.0)
        ids = s.moe.topk_ids[:, :b.k].long()
        if b.mode == 0:
            w = torch.softmax(z.gather(1, ids), 1) if b.renormalize else torch.softmax(z, 1).gather(1, ids)
        else:
            w = torch.sigmoid(z.gather(1, ids))
            w = w / w.sum(1, keepdim=True) if b.renormalize else w
        w = torch.cat([b.router_scale * w, torch.ones(len(x), b.n_shared, dtype=F64, device=DEV)], 1)
        ids = s.moe.topk_ids.long()
        W13, W2 = p["W13"][ids], p["W2"][ids]  # [T, slots, ...]: small sizes
        hh = torch.einsum("th,tjih->tji", h, W13)
        act = torch.nn.functional.silu(hh[..., :b.I]) * hh[..., b.I:]
        y = (torch.einsum("tji,tjhi->tjh", act, W2) * w.unsqueeze(-1)).sum(1)
        u = rms(y, b.eps) * p["gamma_out"]
        x = x + b.scale * (u * p["gate"] if "gate" in p else u)
    return x, (x * dout64).sum()


CASES = [dict(), dict(ns=1, k=1), dict(mode=1, router_scale=2.5), dict(renormalize=False, bias=True), dict(n=3, E=1, k=1)]


@pytest.mark.parametrize("kw", CASES)
@pytest.mark.parametrize("T", [1, 37])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_against_autograd(S, dtype, T, kw):
    stack, rnd = make(S, dtype, seed=T, **kw)
    x, dout = rnd(T, 136).to(dtype), rnd(T, 136).to(dtype)
    out, saved = stack.forward(x)
    dx = stack.backward(dout, saved)
    blocks64 = [{n: t.to(F64).requires_grad_() for n, t in b.parameters().items()} for b in stack.blocks]
    x64 = x.to(F64).requires_grad_()
    ref, loss = reference(stack, saved, x64, dout.to(F64), blocks64)
    loss.backward()
    # A block is a chain of about 16 stages forward and backward (norm, router, products, sums, join);
    # each is off by at most its type's half step, and for fp32 by its sums of up to 2I + H = 280
    # terms, relative to the norm of its result. Errors pass through later blocks with about the gain
    # that values do, so the relative errors of n blocks add: 16 n (half step + 280 * 2^-24).
    n = len(stack.blocks)
    tol = 16 * n * ((2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) + 280 * 2.0 ** -24)

    def near(got, want, what):
        scale = want.norm()
        assert torch.isfinite(got).all(), what
        # a gradient that is zero but for cancellation (one expert: the weights do not move) is held
        # to the size of what cancels, at most that of the incoming gradient
        ref_size = max(scale.item(), 1e-3 * dout.to(F64).norm().item())
        assert (got.to(F64) - want).norm() <= tol * ref_size, f"{what}: {(got.to(F64) - want).norm() / ref_size:.3g} > {tol:.3g}"
    near(out, ref.detach(), "out")
    near(dx, x64.grad, "dx")
    for i, (g, p) in enumerate(zip(stack.grads, blocks64)):
        for name, t in p.items():
            near(g[name], t.grad, f"block {i} {name}")
    # a second backward pass adds the same again
    before = {n_: t.clone() for n_, t in stack.grads[0].items()}
    stack.backward(dout, saved)
    for name, t in before.items():
        near(stack.grads[0][name], 2 * t.to(F64), f"twice {name}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_block_norms_with_its_own_eps(S, dtype):
    """Blocks of different eps, all of the size of a row's mean square, two of them equal."""
    stack, rnd = make(S, dtype, seed=3, n=4)
    for b, eps in zip(stack.blocks, (2.0, 0.25, 0.25, 1e-6)):
        b.eps = eps
    x, dout = rnd(37, 136).to(dtype), rnd(37, 136).to(dtype)
    out, saved = stack.forward(x)
    dx = stack.backward(dout, saved)
    blocks64 = [{n: t.to(F64).requires_grad_() for n, t in b.parameters().items()} for b in stack.blocks]
    x64 = x.to(F64).requires_grad_()
    ref, loss = reference(stack, saved, x64, dout.to(F64), blocks64)
    loss.backward()
    # as for the gradients above: 16 stages a block, each off by its type's half step and fp32's sums
    tol = 16 * 4 * ((2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) + 280 * 2.0 ** -24)
    pairs = [("out", out, ref.detach()), ("dx", dx, x64.grad)]
    pairs += [(f"block {i} {n}", g[n], t.grad) for i, (g, p) in enumerate(zip(stack.grads, blocks64))
              for n, t in p.items()]
    for what, got, want in pairs:
        assert (got.to(F64) - want).norm() <= tol * want.norm(), what


def test_forward_agrees_with_the_inference_layer(S):
    """y of one block against moe_forward on the same normed input (other kernels, bf16)."""
    from routing_grouped_gemm_router_gb300 import training as ops
    from routing_grouped_gemm_router_gb300.layer import MoELayer
    stack, rnd = make(S, torch.bfloat16, n=1, H=512, I=384, E=16, k=4)
    b = stack.blocks[0]
    for T in (1, 200):
        h, _ = ops.block_norm(rnd(T, 512).to(torch.bfloat16), b.gamma_in)
        y, s = b.moe(h)
        layer = MoELayer(b.Wg, b.W13, b.W2, b.k)
        want = layer(h)
        assert torch.equal(layer.intermediates(T)["topk_ids"], s.topk_ids)
        # act, ys (weighted there before rounding, here after) and y are rounded on both sides
        assert (y.to(F64) - want.to(F64)).norm() <= 6 * 2.0 ** -8 * want.to(F64).norm()


def test_a_captured_step_replays_with_new_inputs(S):
    stack, rnd = make(S, torch.bfloat16)
    x, dout = rnd(64, 136).to(torch.bfloat16), rnd(64, 136).to(torch.bfloat16)

    def step():
        stack.zero_grad()
        out, saved = stack.forward(x)
        return [out, stack.backward(dout, saved)] + [t for g in stack.grads for t in g.values()]
    eager_kept = step()  # results of an eager pass stay alive through the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    new = rnd(64, 136).to(torch.bfloat16)
    x.copy_(new)
    want = [t.clone() for t in step()]
    x.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert all(torch.isfinite(t.float()).all() for t in eager_kept)


def test_the_example_learns():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import train_sparse_stack as ex
    eager = ex.train(steps=12)
    assert eager[-1] < 0.9 * eager[0]
    assert ex.train(steps=12, graph=True) == eager  # the same bits from replays
