"""A trainable stack of sparse blocks from token ids, on the operators of ``training``:

    x <- dropout(embed_scale * table[tokens])
    x <- x + scale * dropout(MoE(layer_norm(x)))      for every block,
    h  = layer_norm(x),

with the balance and z losses of every block's router. Forward and backward are explicit calls, as in
``sparse_block``: ``backward`` takes the gradient of h and the weights of the router's losses, and adds
to gradients that the stack owns. A whole step can be captured in a CUDA graph; ``rng`` holds the
seed and the step's stream on the device, and a program writes the stream between steps.
"""
from __future__ import annotations

from typing import List, NamedTuple, Optional

import torch

from . import _lib as L
from . import training as ops
from .sparse_block import BalanceGrads, MoESaved, SparseLayer, _fits


class TokenBlock(SparseLayer):
    """A SparseLayer and the layer norm before it: gamma[H], and beta[H] or None, fp32."""

    names = ("Wg", "W13", "W2", "gamma", "beta")

    def __init__(self, Wg, W13, W2, gamma, beta, k: int, scale: float = 1.0, mode: int = L.MOE_ROUTE_SOFTMAX,
                 renormalize: bool = True, router_scale: float = 1.0, n_group: int = 1, topk_group: int = 1,
                 logit_bias=None, select_bias=None, n_shared: int = 0):
        super().__init__(Wg, W13, W2, k, mode, renormalize, router_scale, n_group, topk_group, logit_bias,
                         select_bias, n_shared)
        _check_norm("", gamma, beta, self.H, Wg.device)
        self.gamma, self.beta, self.scale = gamma, beta, scale


def _check_norm(suffix, gamma, beta, H, device):
    _fits("gamma" + suffix, gamma, (H,), torch.float32, device)
    if beta is not None:
        _fits("beta" + suffix, beta, (H,), torch.float32, device)


class TokenBlockSaved(NamedTuple):
    moe: MoESaved
    balance: ops.BalanceLoss
    out: torch.Tensor   # after the join
    mean: torch.Tensor  # of its rows, for the next norm
    rstd: torch.Tensor


class TokenStackSaved(NamedTuple):
    tokens: torch.Tensor  # these, rng, offsets and mask: as they were in the forward pass
    rng: torch.Tensor
    x: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor
    blocks: List[TokenBlockSaved]
    offsets: Optional[torch.Tensor]
    mask: Optional[torch.Tensor]
    p: float  # of the forward pass's dropout


class TokenStack:
    """table[V, H] in the blocks' type; gamma_final[H], and beta_final[H] or None, fp32; p: dropout after the
    embedding and in every join (set to 0 for a pass without; a backward pass takes its forward pass's); seed: of
    the random numbers."""

    def __init__(self, table, blocks: List[TokenBlock], gamma_final, beta_final=None, embed_scale: float = 1.0,
                 p: float = 0.0, seed: int = 0, eps: float = 1e-5):
        if not blocks:
            raise ValueError("blocks: at least one is needed")
        if not 0.0 <= p < 1.0:
            raise ValueError(f"p: {p}, expected 0 <= p < 1")
        first = blocks[0]
        self.H, dtype, device = first.H, first.Wg.dtype, first.Wg.device
        _fits("table", table, (None, self.H), dtype, device)
        for i, b in enumerate(blocks):
            _fits(f"blocks[{i}].Wg", b.Wg, (None, self.H), dtype, device)
        _check_norm("_final", gamma_final, beta_final, self.H, device)
        self.table, self.blocks = table, list(blocks)
        self.gamma_final, self.beta_final = gamma_final, beta_final
        self.embed_scale, self.p, self.eps = embed_scale, p, eps
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=device)
        own = {"table": table, "gamma_final": gamma_final, "beta_final": beta_final}
        self._own = {n: t for n, t in own.items() if t is not None}
        zeros = lambda ts: {n: torch.zeros_like(t, dtype=torch.float32) for n, t in ts.items()}  # noqa: E731
        self.grads = zeros(self._own)
        self.block_grads = [zeros(b.parameters()) for b in self.blocks]

    def parameters(self):
        """name -> tensor of the stack's own; the blocks have theirs."""
        return dict(self._own)

    def zero_grad(self):
        for g in [self.grads, *self.block_grads]:
            for t in g.values():
                t.zero_()

    def _norm_after(self, i):
        """gamma and beta of the norm that reads block i's output, and their gradients' dict and names."""
        if i + 1 < len(self.blocks):
            b = self.blocks[i + 1]
            return b.gamma, b.beta, self.block_grads[i + 1], "gamma", "beta"
        return self.gamma_final, self.beta_final, self.grads, "gamma_final", "beta_final"

    def forward(self, tokens, offsets=None, mask=None):
        """(h[T, H], losses[blocks, 2], saved) for token ids [T], int32 or int64. offsets and mask: the packed
        sequences and the tokens that take part in the router's losses (``balance_loss``). The caller's
        tensors may be written once the call has returned."""
        rng = self.rng.clone()  # the backward pass draws the same numbers, whatever is written meanwhile
        x = ops.embed(tokens, self.table, self.embed_scale)
        if self.p:
            x = ops.dropout(x, self.p, rng, 0)
        first = self.blocks[0]
        h, mean, rstd = ops.layer_norm(x, first.gamma, first.beta, self.eps)
        saved, out = [], x
        for i, b in enumerate(self.blocks):
            y, s = b.moe(h)
            bal = ops.balance_loss(s.logits, s.topk_ids, b.mode, b.logit_bias, b.n_shared, offsets, mask)
            gamma, beta = self._norm_after(i)[:2]
            j = ops.dropout_join(out, y, self.p, rng, 1 + i, b.scale, gamma, beta, self.eps)
            out, h = j.out, j.h
            saved.append(TokenBlockSaved(s, bal, out, j.mean, j.rstd))
        losses = torch.stack([s.balance.losses for s in saved])
        # copies: a program may fill its buffers with the next batch before the backward pass
        inputs = [None if t is None else t.clone() for t in (tokens, offsets, mask)]
        return h, losses, TokenStackSaved(inputs[0], rng, x, mean, rstd, saved, *inputs[1:], self.p)

    __call__ = forward

    def backward(self, dh, saved: TokenStackSaved, dlosses=None):
        """Adds the gradients of all parameters to ``grads`` and ``block_grads``. dh: the gradient of h;
        dlosses: fp32 [2], the weight of every block's balance and z loss in the total (None: neither)."""
        dres = None
        for i in reversed(range(len(self.blocks))):
            b, s = self.blocks[i], saved.blocks[i]
            gamma, beta, grads, gname, bname = self._norm_after(i)
            j = ops.dropout_join_backward(dres, saved.p, saved.rng, 1 + i, b.scale, dh, s.out, gamma, s.mean,
                                          s.rstd, beta is not None)
            grads[gname].add_(j.dgamma_next)
            if beta is not None:
                grads[bname].add_(j.dbeta_next)
            bal = None if dlosses is None else BalanceGrads(dlosses, s.balance, saved.offsets, saved.mask)
            dres, dh = j.dx, b.moe_backward(j.dy, s.moe, self.block_grads[i], bal)
        first, g = self.blocks[0], self.block_grads[0]
        n = ops.layer_norm_backward(dh, saved.x, first.gamma, saved.mean, saved.rstd, dres, first.beta is not None)
        g["gamma"].add_(n.dgamma)
        if first.beta is not None:
            g["beta"].add_(n.dbeta)
        dx = ops.dropout(n.dx, saved.p, saved.rng, 0) if saved.p else n.dx
        ops.embed_backward(dx, saved.tokens, self.table.shape[0], self.embed_scale, out=self.grads["table"],
                           accumulate=True)
