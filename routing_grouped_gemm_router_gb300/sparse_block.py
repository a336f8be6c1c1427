"""Trainable stacks of sparse blocks on the operators of ``training``. SparseStack:

    x <- x + scale * gate . norm(MoE(norm(x)))        for every block,

a norm before and after the MoE layer (RMS, fp32 weights), an optional gate, a residual scale.
TokenStack (token_stack.py) trains blocks x <- x + scale * dropout(MoE(layer_norm(x))) from token ids.
Forward and backward are explicit calls: ``forward`` keeps what the backward pass needs,
``backward`` takes the gradient of the output and adds to gradients that the stack owns, so a
whole step allocates from PyTorch's pool only and can be captured in a CUDA graph.

Everything but two small dense products runs in the library's kernels; the router's weight and
input gradients (dlogits^T h and dlogits Wg) are plain torch products.
"""
from __future__ import annotations

from typing import List, NamedTuple, Optional

import torch

from . import _lib as L
from . import training as ops


def _fits(name, t, shape, dtype, device):
    """ValueError by name unless t is a contiguous tensor of this shape (None: any extent), type and
    device: the router's entry point takes bare addresses and would misread any other."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != len(shape) or any(d is not None and d != n for d, n in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected "
                         f"({', '.join('any' if d is None else str(d) for d in shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous (strides {t.stride()})")
    if t.device != device:
        raise ValueError(f"{name}: is on {t.device}, expected {device}")


class SparseLayer:
    """Router and experts of one block: Wg[E, H], W13[E', 2I, H], W2[E', H, I] all in bf16 or all in fp32
    (E' = E + n_shared: shared experts follow the routed ones); logit_bias, select_bias: None or fp32
    [E]. All contiguous, on one device; anything else raises ValueError."""

    def __init__(self, Wg, W13, W2, k: int, mode: int = L.MOE_ROUTE_SOFTMAX, renormalize: bool = True,
                 router_scale: float = 1.0, n_group: int = 1, topk_group: int = 1,
                 logit_bias=None, select_bias=None, n_shared: int = 0):
        if not isinstance(Wg, torch.Tensor) or Wg.dim() != 2 or Wg.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("Wg: a bfloat16 or float32 tensor [E, H] is needed")
        for name, t in (("W13", W13), ("W2", W2)):
            _fits(name, t, (None, None, None), Wg.dtype, Wg.device)
        if W13.shape[0] != Wg.shape[0] + n_shared or W2.shape[0] != W13.shape[0]:
            raise ValueError(f"W13, W2: {W13.shape[0]} and {W2.shape[0]} experts, expected "
                             f"{Wg.shape[0]} routed and {n_shared} shared ones")
        if W13.shape[1] != 2 * W2.shape[2] or W13.shape[2] != Wg.shape[1] or W2.shape[1] != Wg.shape[1]:
            raise ValueError(f"W13 {tuple(W13.shape)}, W2 {tuple(W2.shape)}, Wg {tuple(Wg.shape)}: "
                             "extents do not belong together")
        self.Wg, self.W13, self.W2 = Wg, W13, W2
        self.E, self.H = Wg.shape
        self.I, self.k, self.n_shared = W2.shape[2], k, n_shared
        self.mode, self.renormalize, self.router_scale = mode, renormalize, router_scale
        self.n_group, self.topk_group = n_group, topk_group
        self.logit_bias, self.select_bias = logit_bias, select_bias
        self._check_router()

    names = ("Wg", "W13", "W2")  # of the tensors that train

    def _check_router(self):
        """What moe_route is given by address besides the tokens."""
        _fits("Wg", self.Wg, (self.E, self.H), self.W13.dtype, self.W13.device)
        for name, t in (("logit_bias", self.logit_bias), ("select_bias", self.select_bias)):
            if t is not None:
                _fits(name, t, (self.E,), torch.float32, self.Wg.device)

    def _check_tokens(self, name, x):
        """Token rows that go with the block's weights, on the current CUDA device."""
        _fits(name, x, (None, self.H), self.Wg.dtype, self.Wg.device)
        if not x.is_cuda or x.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name}: is on {x.device}, has to be on the current CUDA device")

    def parameters(self):
        """name -> tensor, of those that train."""
        p = {n: getattr(self, n) for n in self.names}
        return {n: t for n, t in p.items() if t is not None}

    def route(self, h):
        """(logits, topk_ids, topk_w) of ``moe_route``; ids and weights hold k + n_shared slots."""
        self._check_router()  # attributes can have been replaced
        self._check_tokens("h", h)
        T, kk = h.shape[0], self.k + self.n_shared
        logits = torch.empty(T, self.E, dtype=torch.float32, device=h.device)
        ids = torch.empty(T, kk, dtype=torch.int32, device=h.device)
        w = torch.empty(T, kk, dtype=torch.float32, device=h.device)
        cfg = L.make_config(T, self.H, self.I, self.E, self.k, L.MOE_BF16 if h.dtype == torch.bfloat16 else L.MOE_F32, self.mode,
                            self.renormalize, self.router_scale, self.n_group, self.topk_group,
                            self.logit_bias, self.select_bias, n_shared=self.n_shared)
        L.moe_route(cfg, h, self.Wg, logits, ids, w)
        return logits, ids, w

    def moe(self, h):
        """(y, saved): the routed experts' outputs for the normed input h."""
        logits, ids, w = self.route(h)
        table = ops.sort_tokens(ids, self.E + self.n_shared)
        xs, pos = ops.permute(h, ids, table.sorted_ids, self.E + self.n_shared)
        h13, act = ops.expert_up(xs, self.W13, table.counts)
        ys = ops.expert_down(act, self.W2, table.counts)
        return ops.unpermute(ys, pos, w), MoESaved(h, logits, ids, w, table.sorted_ids, table.counts, pos,
                                                   xs, h13, ys)

    def moe_backward(self, dy, s: "MoESaved", grads: dict, balance: Optional["BalanceGrads"] = None):
        """dh; gradients of Wg, W13 and W2 are added to grads (fp32 tensors of their shapes). balance: the
        router's losses that go into the total, if any."""
        dys, dw = ops.unpermute_backward(dy, s.ys, s.sorted_ids, s.row_pos, s.topk_w)
        dh13, act = ops.expert_down_backward(dys, self.W2, s.h13, s.counts)
        ops.expert_weight_grad(dys, act, s.counts, out=grads["W2"], accumulate=True)
        ops.expert_weight_grad(dh13, s.xs, s.counts, out=grads["W13"], accumulate=True)
        dh = ops.permute_backward(ops.expert_up_backward(dh13, self.W13, s.counts), s.row_pos)
        dlogits = ops.route_backward(s.logits, s.topk_ids, dw, self.mode, self.renormalize,
                                     self.router_scale, self.logit_bias, self.n_shared)
        if balance is not None:
            ops.balance_loss_backward(balance.dlosses, s.logits, balance.saved, self.k, self.mode, self.logit_bias,
                                      balance.offsets, balance.mask, dlogits=dlogits)
        grads["Wg"].addmm_(dlogits.T, s.h.float())
        # with bf16 weights dlogits is rounded to bf16 here, as the product of two bf16 matrices takes it:
        # each term is then off by at most 2^-8 of itself, as h and Wg are, and the sum over experts is fp32
        return torch.addmm(dh, dlogits.to(dh.dtype), self.Wg)


class SparseBlock(SparseLayer):
    """A SparseLayer and the norms around it: gamma_in[H] and gamma_out[H] fp32; gate: None or fp32 [H], the
    same for all tokens (where the number of tokens is fixed, any gate of block_join). All contiguous, on
    one device; anything else raises ValueError."""

    names = ("Wg", "W13", "W2", "gamma_in", "gamma_out", "gate")

    def __init__(self, Wg, W13, W2, gamma_in, gamma_out, k: int, gate=None, scale: float = 1.0,
                 mode: int = L.MOE_ROUTE_SOFTMAX, renormalize: bool = True,
                 router_scale: float = 1.0, n_group: int = 1, topk_group: int = 1,
                 logit_bias=None, select_bias=None, n_shared: int = 0, eps: float = 1e-6):
        super().__init__(Wg, W13, W2, k, mode, renormalize, router_scale, n_group, topk_group, logit_bias,
                         select_bias, n_shared)
        self.gamma_in, self.gamma_out, self.gate = gamma_in, gamma_out, gate
        self.scale, self.eps = scale, eps
        for name, t in (("gamma_in", gamma_in), ("gamma_out", gamma_out)):
            _fits(name, t, (self.H,), torch.float32, Wg.device)
        if gate is not None:
            rank = gate.dim() if isinstance(gate, torch.Tensor) else 1
            full = rank == 2 and gate.shape[1] != 1
            _fits("gate", gate, (self.H,) if rank == 1 else (None, self.H if full else 1),
                  Wg.dtype if full else torch.float32, Wg.device)


class BalanceGrads(NamedTuple):
    """The router's losses in a total: their weights (fp32 [2] on the device), what ``balance_loss`` returned and
    the sequences and tokens that it was given."""
    dlosses: torch.Tensor
    saved: ops.BalanceLoss
    offsets: Optional[torch.Tensor] = None
    mask: Optional[torch.Tensor] = None


class MoESaved(NamedTuple):
    h: torch.Tensor
    logits: torch.Tensor
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    sorted_ids: torch.Tensor
    counts: torch.Tensor
    row_pos: torch.Tensor
    xs: torch.Tensor
    h13: torch.Tensor
    ys: torch.Tensor


class BlockSaved(NamedTuple):
    moe: MoESaved
    y: torch.Tensor
    rstd_y: torch.Tensor
    out: torch.Tensor
    rstd_out: Optional[torch.Tensor]  # of the next block's norm


class StackSaved(NamedTuple):
    x: torch.Tensor
    rstd: torch.Tensor
    blocks: List[BlockSaved]


class SparseStack:
    """Blocks in sequence. A block's residual join also takes the next block's norm, where both blocks
    have the same eps."""

    def __init__(self, blocks: List[SparseBlock]):
        if not blocks:
            raise ValueError("blocks: at least one is needed")
        self.blocks = list(blocks)
        for i, b in enumerate(self.blocks):  # every block's tokens are the first one's
            _fits(f"blocks[{i}].Wg", b.Wg, (None, self.blocks[0].H), self.blocks[0].Wg.dtype,
                  self.blocks[0].Wg.device)
        self.grads = [{n: torch.zeros_like(t, dtype=torch.float32) for n, t in b.parameters().items()}
                      for b in self.blocks]

    def zero_grad(self):
        for g in self.grads:
            for t in g.values():
                t.zero_()

    def forward(self, x):
        """(out[T, H], saved) for x[T, H], which saved holds by reference: it stays as it is until ``backward``."""
        first = self.blocks[0]
        first._check_tokens("x", x)
        h, rstd = ops.block_norm(x, first.gamma_in, first.eps)
        saved, out = [], x
        for i, b in enumerate(self.blocks):
            y, s = b.moe(h)
            nxt = self.blocks[i + 1] if i + 1 < len(self.blocks) else None
            fused = nxt is not None and nxt.eps == b.eps  # block_join takes both its norms with one eps
            j = ops.block_join(out, y, b.gamma_out, b.gate, b.scale, nxt.gamma_in if fused else None, b.eps)
            out, h, rstd_out = j.out, j.h, j.rstd_out
            if nxt is not None and not fused:
                h, rstd_out = ops.block_norm(out, nxt.gamma_in, nxt.eps)
            saved.append(BlockSaved(s, y, j.rstd_y, out, rstd_out))
        return out, StackSaved(x, rstd, saved)

    __call__ = forward

    def backward(self, dout, saved: StackSaved):
        """dx; the gradients of every block's parameters are added to ``grads``."""
        dres, dh = dout, None
        for i in reversed(range(len(self.blocks))):
            b, g, s = self.blocks[i], self.grads[i], saved.blocks[i]
            nxt = {}
            if dh is not None:
                nxt = dict(dh=dh, out=s.out, gamma_next=self.blocks[i + 1].gamma_in, rstd_out=s.rstd_out)
            j = ops.block_join_backward(dres, s.y, b.gamma_out, s.rstd_y, b.gate, b.scale, **nxt)
            g["gamma_out"].add_(j.dgamma)
            if b.gate is not None:
                g["gate"].add_(j.dgate)
            if dh is not None:
                self.grads[i + 1]["gamma_in"].add_(j.dgamma_next)
            dres, dh = j.dx, b.moe_backward(j.dy, s.moe, g)
        first = self.blocks[0]
        dx, dgamma = ops.block_norm_backward(dh, saved.x, first.gamma_in, saved.rstd, dres)
        self.grads[0]["gamma_in"].add_(dgamma)
        return dx
