"""Trains a small stack of sparse blocks to predict the next token of synthetic sequences.

    python examples/train_token_stack.py [--steps 60] [--graph]

Packed sequences of random lengths, in which every token follows from the one before by a fixed table
most of the time. Every step is a forward pass (embedding, layer norms, dropout, experts, the
router's balance and z losses), a cross entropy against the embedding's own table, the backward pass
and plain gradient descent with momentum on fp32 copies of the weights. --graph captures the whole
step in a CUDA graph and replays it; the step's number goes into the random numbers' stream.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from routing_grouped_gemm_router_gb300.token_stack import TokenBlock, TokenStack  # noqa: E402


def make_stack(seed, V, n_blocks=2, H=256, I=192, E=16, k=4, p=0.1, dtype=torch.bfloat16, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device=device) * std).to(dtype)  # noqa: E731
    ones, zeros = (lambda: torch.ones(H, device=device)), (lambda: torch.zeros(H, device=device))
    blocks = [TokenBlock(rnd(E, H, std=H ** -0.5), rnd(E, 2 * I, H, std=H ** -0.5), rnd(E, H, I, std=I ** -0.5),
                         ones(), zeros(), k) for _ in range(n_blocks)]
    return TokenStack(rnd(V, H, std=H ** -0.5), blocks, ones(), zeros(), embed_scale=H ** 0.5, p=p, seed=seed)


def batch(g, T, V, follows, n_sequences):
    """(tokens, offsets): ragged sequences packed into T tokens."""
    tokens = torch.randint(0, V, (T,), generator=g)
    free = torch.rand(T, generator=g) < 0.1
    cuts = torch.randint(1, T, (n_sequences - 1,), generator=g).sort().values
    offsets = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])])
    free[offsets[:-1]] = True
    for t in range(1, T):
        if not free[t]:
            tokens[t] = follows[tokens[t - 1]]
    return tokens, offsets.to(torch.int32)


def train(steps=60, T=1024, V=384, lr=0.5, momentum=0.9, graph=False, seed=0, balance=1e-2, z=1e-3):
    """Cross entropies, first to last."""
    stack = make_stack(seed, V)
    params = [(t, g[n], t.float().clone(), torch.zeros_like(t, dtype=torch.float32))
              for owner, g in [(stack, stack.grads), *zip(stack.blocks, stack.block_grads)]
              for n, t in owner.parameters().items()]
    tokens = torch.zeros(T, dtype=torch.int64, device="cuda")
    offsets = torch.zeros(9, dtype=torch.int32, device="cuda")
    loss = torch.zeros((), device="cuda")
    up = torch.tensor([balance, z], device="cuda")

    def step():
        stack.zero_grad()
        h, _, saved = stack.forward(tokens, offsets)
        # the next token, where it is of the same sequence
        at = torch.arange(1, T, device="cuda")
        inside = (at[:, None] != offsets[None, 1:-1]).all(1)
        logits = (h[:-1] @ stack.table.T).float()
        logp = logits - logits.logsumexp(1, keepdim=True)
        weight = inside.float() / inside.sum()
        loss.copy_(-(logp.gather(1, tokens[1:, None])[:, 0] * weight).sum())
        d = logp.exp()
        d.scatter_add_(1, tokens[1:, None], torch.full((T - 1, 1), -1.0, device="cuda"))
        d = (d * weight[:, None]).to(h.dtype)
        stack.grads["table"].add_(d.T.float() @ h[:-1].float())
        dh = torch.zeros_like(h)
        dh[:-1] = d @ stack.table
        stack.backward(dh, saved, up)
        for t, g, master, velocity in params:
            velocity.mul_(momentum).add_(g)
            master.add_(velocity, alpha=-lr)
            t.copy_(master)

    g = torch.Generator()
    g.manual_seed(seed)
    follows = torch.randperm(V, generator=g)
    losses, captured = [], None
    for i in range(steps):
        new_tokens, new_offsets = batch(g, T, V, follows, 8)
        tokens.copy_(new_tokens)
        offsets.copy_(new_offsets)
        stack.rng[1] = i
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
            print(f"step {i:4d}  cross entropy {v:.5f}")
