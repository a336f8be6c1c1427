"""Trains a small stack of sparse blocks to follow another one, on synthetic tokens.

    python examples/train_sparse_stack.py [--steps 60] [--graph]

Every step is a forward pass, the gradient of a mean squared error, the backward pass through the
framework's training operators and plain gradient descent with momentum on fp32 copies of the
weights. --graph captures the whole step in a CUDA graph and replays it.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from routing_grouped_gemm_router_gb300.sparse_block import SparseBlock, SparseStack  # noqa: E402


def make_stack(seed, n_blocks=2, H=512, I=384, E=16, k=4, dtype=torch.bfloat16, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device=device) * std).to(dtype)  # noqa: E731
    return SparseStack([
        SparseBlock(rnd(E, H, std=H ** -0.5), rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5),
                    torch.ones(H, device=device), torch.ones(H, device=device), k,
                    gate=torch.full((H,), 0.5, device=device), scale=0.5)
        for _ in range(n_blocks)])


def train(steps=60, T=1024, lr=2.0, momentum=0.9, graph=False, seed=0):
    """Losses, first to last."""
    teacher, student = make_stack(seed + 1), make_stack(seed + 2)
    H = student.blocks[0].H
    # fp32 copies that the optimiser moves; the blocks' own weights follow them
    params = [(b, n, t, t.float().clone(), torch.zeros_like(t, dtype=torch.float32))
              for b in student.blocks for n, t in b.parameters().items()]
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    loss = torch.zeros((), device="cuda")

    def step():
        want, _ = teacher.forward(x)
        out, saved = student.forward(x)
        diff = out.float() - want.float()
        loss.copy_(diff.square().mean())
        student.zero_grad()
        student.backward((diff * (2.0 / T)).to(out.dtype), saved)
        grads = (g[n] for b, g in zip(student.blocks, student.grads) for n in b.parameters())
        for (_, _, t, master, velocity), g in zip(params, grads):
            velocity.mul_(momentum).add_(g, alpha=1.0 / H)
            master.add_(velocity, alpha=-lr)
            t.copy_(master)

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    losses, captured = [], None
    for i in range(steps):
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        if graph and i == 2:  # the first steps ran eagerly: everything is loaded and allocated
            torch.cuda.synchronize()
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        if captured is not None:
            captured.replay()
        else:
            step()
        losses.append(float(loss))
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--graph", action="store_true")
    a = ap.parse_args()
    for i, v in enumerate(train(a.steps, graph=a.graph)):
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {v:.5f}")
