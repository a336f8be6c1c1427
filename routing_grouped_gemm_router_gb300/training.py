"""The operators that train a sparse block and the stack around it, on tensors: checks of arguments,
output and workspace allocation (PyTorch's caching allocator, current stream) around the C entry
points of ``include/moe_train.h`` and ``moe_stack.h``, which say what each computes. The checks and calls are compiled
(``csrc/binding.cpp``, ``binding_stack.cpp``); a tensor that does not fit raises ``ValueError`` by its name, a status of the
library ``MoeError``.

Every function takes contiguous tensors of the current CUDA device, enqueues on the current
stream, returns new tensors, and never synchronises: a whole step, backward pass included, can be
captured in a CUDA graph. The backward functions are called explicitly with what the forward
ones returned; nothing here builds an autograd graph.

Rows sorted by expert sit in buffers of ``buffer_rows(T, k, E)`` rows in which every expert's
run is padded to 16 rows; rows of no slot are zeros.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib as L
from . import _native as C
from . import _native_stack as S

C.set_error(L.MoeError)
S.set_error(L.MoeError)


def buffer_rows(T: int, k: int, E: int) -> int:
    """Rows of the expert-sorted buffers of T tokens with k slots each over E experts."""
    return L.moe_max_padded_rows(T, k, E, L.MOE_TRAIN_BLOCK)


# ------------------------------------------------------------------------------- dispatch
class SortedTokens(NamedTuple):
    sorted_ids: torch.Tensor       # int32 [rows]: slot of each row, T*k where there is none
    expert_ids: torch.Tensor       # int32 [rows / 16]: expert of each 16-row block, -1 past the end
    num_post_padded: torch.Tensor  # int32 [1]: rows up to the end of the last run
    counts: torch.Tensor           # int32 [E]: slots of each expert


def sort_tokens(topk_ids, E: int) -> SortedTokens:
    """The table of the routed slots sorted by expert (``moe_align`` with 16-row blocks).
    Ids outside [0, E) are dropped (and recorded in the device status)."""
    return SortedTokens._make(C.sort_tokens(topk_ids, E))


def permute(x, topk_ids, sorted_ids, E: int):
    """(xs[rows, H], row_pos[T, k]): token rows copied to their slots' rows; -1 for dropped slots."""
    return C.permute(x, topk_ids, sorted_ids, E)


def permute_backward(dxs, row_pos):
    """dx[T, H]: the gradients of a token's rows summed over its slots."""
    return C.permute_backward(dxs, row_pos)


def unpermute(ys, row_pos, topk_w):
    """out[T, H]: the rows of a token's slots, weighted and summed."""
    return C.unpermute(ys, row_pos, topk_w)


def unpermute_backward(dout, ys, sorted_ids, row_pos, topk_w):
    """(dys[rows, H], dtopk_w[T, k]) of ``unpermute``."""
    return C.unpermute_backward(dout, ys, sorted_ids, row_pos, topk_w)


# -------------------------------------------------------------------------------- experts
def expert_up(xs, W13, counts):
    """(h13[rows, 2I], act[rows, I]): gate and up projections (fp32, kept for the backward pass) and
    silu(gate) * up of every expert's rows."""
    return C.expert_up(xs, W13, counts)


def expert_down(act, W2, counts):
    """ys[rows, H]: the down projection of every expert's rows, without the router weight."""
    return C.expert_down(act, W2, counts)


def expert_down_backward(dys, W2, h13, counts):
    """(dh13[rows, 2I], act[rows, I]): the gradient through the down projection and the SwiGLU, and
    the activations computed again for the gradient of W2."""
    return C.expert_down_backward(dys, W2, h13, counts)


def expert_up_backward(dh13, W13, counts):
    """dxs[rows, H]: the gradient through the gate and up projections."""
    return C.expert_up_backward(dh13, W13, counts)


def expert_weight_grad(dy, a, counts, out: Optional[torch.Tensor] = None,
                       out_dtype: Optional[torch.dtype] = None, accumulate: bool = False):
    """dW[E, M, N] = dy_e^T a_e over every expert's rows: W2's gradient from (dys, act), W13's from
    (dh13, xs). `out` is overwritten, or added to with `accumulate`; otherwise a new tensor of
    out_dtype (default: dy's) is returned."""
    return C.expert_weight_grad(dy, a, counts, out, out_dtype, accumulate)


# -------------------------------------------------------------------- norms around the block
def block_norm(x, gamma, eps: float = 1e-6, offset: float = 0.0):
    """(h, rstd): x * rstd * (offset + gamma), rstd = (mean(x^2) + eps)^-1/2 of each row."""
    return C.block_norm(x, gamma, eps, offset)


def block_norm_backward(dh, x, gamma, rstd, dres=None, offset: float = 0.0):
    """(dx, dgamma) of ``block_norm``; dres, the gradient that reaches x past the norm, is added."""
    return C.block_norm_backward(dh, x, gamma, rstd, dres, offset)


class Joined(NamedTuple):
    out: torch.Tensor
    rstd_y: torch.Tensor
    h: Optional[torch.Tensor]         # the next block's normed input
    rstd_out: Optional[torch.Tensor]


def block_join(x, y, gamma, gate=None, scale: float = 1.0, gamma_next=None, eps: float = 1e-6,
               offset: float = 0.0) -> Joined:
    """out = x + scale * gate * norm(y; gamma), and h = norm(out; gamma_next) of the same pass, both
    norms with this eps and offset (a next norm with others: gamma_next None, then block_norm of out).
    gate: None, fp32 [H] (a channel), fp32 [T, 1] (a token) or [T, H] of x's dtype."""
    return Joined._make(C.block_join(x, y, gamma, gate, scale, gamma_next, eps, offset))


class JoinGrads(NamedTuple):
    dx: torch.Tensor
    dy: torch.Tensor
    dgamma: torch.Tensor
    dgamma_next: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


def block_join_backward(dres, y, gamma, rstd_y, gate=None, scale: float = 1.0, dh=None, out=None,
                        gamma_next=None, rstd_out=None, offset: float = 0.0) -> JoinGrads:
    """Gradients of ``block_join``. dres: the gradient of `out` from past the next norm (None: no
    such path); dh, out, gamma_next, rstd_out: the next norm's, when the join had one."""
    return JoinGrads._make(C.block_join_backward(dres, y, gamma, rstd_y, gate, scale, dh, out,
                                                 gamma_next, rstd_out, offset))


# --------------------------------------------------------------------------------- router
def route_backward(logits, topk_ids, dtopk_w, mode: int = L.MOE_ROUTE_SOFTMAX,
                   renormalize: bool = True, scale: float = 1.0, logit_bias=None,
                   n_shared: int = 0):
    """dlogits[T, E] from the gradient of ``moe_route``'s topk_w, for the ids it chose."""
    return C.route_backward(logits, topk_ids, dtopk_w, mode, renormalize, scale, logit_bias, n_shared)


# ------------------------------------------------------------------------------ embedding
def embed(tokens, table, scale: float = 1.0):
    """x[T, H] = scale * table[tokens]: tokens int32 or int64 [T], table [V, H]. A token outside [0, V)
    (padding) is a row of zeros."""
    return S.embed(tokens, table, scale)


def embed_backward(dx, tokens, V: int, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, accumulate: bool = False):
    """dtable[V, H] of ``embed``: the gradients of an id's tokens summed in order, the same bits every
    run. `out` is overwritten, or added to with `accumulate` (ids that do not occur are then not
    touched); otherwise a new tensor of out_dtype (default: dx's) is returned."""
    return S.embed_backward(dx, tokens, V, scale, out, out_dtype, accumulate)


# -------------------------------------------------------------- layer norm, dropout, the join
class LayerNormed(NamedTuple):
    h: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor


def layer_norm(x, gamma, beta=None, eps: float = 1e-5) -> LayerNormed:
    """h = (x - mean) * rstd * gamma + beta of each row; gamma and beta fp32 [H]."""
    return LayerNormed._make(S.layer_norm(x, gamma, beta, eps))


class LayerNormGrads(NamedTuple):
    dx: torch.Tensor
    dgamma: torch.Tensor
    dbeta: Optional[torch.Tensor]


def layer_norm_backward(dh, x, gamma, mean, rstd, dres=None, beta: bool = True) -> LayerNormGrads:
    """Gradients of ``layer_norm``; dres, the gradient that reaches x past the norm, is added to dx.
    beta: whether the norm had one (dbeta is None otherwise)."""
    return LayerNormGrads._make(S.layer_norm_backward(dh, x, gamma, mean, rstd, dres, beta))


def dropout(x, p: float, rng=None, site: int = 0, scale: float = 1.0):
    """scale * x[T, H] with every element dropped with probability p and the others over 1 - p. Its own
    gradient: call it on dout with the same p, rng and site.

    rng: int64 [2] on the device, (seed, stream). The mask is a function of seed, stream, site and the
    element's number (a counter-based generator) and is never stored. A program keeps one seed, gives
    every place in a step its own site (0 <= site < 2^32) and every step its own stream, by writing
    rng[1] on the device between steps: a captured step then draws new masks with every replay."""
    return S.dropout(x, p, rng, site, scale)


class DropoutJoined(NamedTuple):
    out: torch.Tensor
    h: Optional[torch.Tensor]     # the next block's normed input
    mean: Optional[torch.Tensor]  # of out's rows
    rstd: Optional[torch.Tensor]


def dropout_join(x, y, p: float = 0.0, rng=None, site: int = 0, scale: float = 1.0, gamma_next=None,
                 beta_next=None, eps: float = 1e-5) -> DropoutJoined:
    """out = x + scale * dropout(y), and with gamma_next h = layer_norm(out; gamma_next, beta_next) of
    the same pass. p, rng, site: see ``dropout`` (rng may be None where p is 0)."""
    return DropoutJoined._make(S.dropout_join(x, y, p, rng, site, scale, gamma_next, beta_next, eps))


class DropoutJoinGrads(NamedTuple):
    dx: torch.Tensor
    dy: torch.Tensor
    dgamma_next: Optional[torch.Tensor]
    dbeta_next: Optional[torch.Tensor]


def dropout_join_backward(dres, p: float = 0.0, rng=None, site: int = 0, scale: float = 1.0, dh=None,
                          out=None, gamma_next=None, mean=None, rstd=None,
                          beta: bool = True) -> DropoutJoinGrads:
    """Gradients of ``dropout_join``. dres: the gradient of `out` from past the next norm (None: no such
    path); dh, out, gamma_next, mean, rstd: the next norm's, when the join had one, and beta whether
    that norm has a bias. Without a next norm dx is dres itself."""
    return DropoutJoinGrads._make(S.dropout_join_backward(dres, p, rng, site, scale, dh, out, gamma_next,
                                                          mean, rstd, beta))


# ------------------------------------------------------------------------- the router's losses
class BalanceLoss(NamedTuple):
    losses: torch.Tensor  # fp32 [2]: balance loss, z loss
    counts: torch.Tensor  # int32 [S, E]: a sequence's slots of every expert
    tokens: torch.Tensor  # int32 [S]: a sequence's tokens that take part
    prob: torch.Tensor    # fp32 [S, E]: mean probability over them
    totals: torch.Tensor  # int32 [2]: sequences with such tokens, such tokens


def balance_loss(logits, topk_ids, mode: int = L.MOE_ROUTE_SOFTMAX, logit_bias=None, n_shared: int = 0,
                 offsets=None, mask=None) -> BalanceLoss:
    """The router's balance loss (mean over sequences of sum_e E counts / (k tokens) * prob), z loss (mean of
    logsumexp(logits)^2) and per-expert counts from what ``moe_route`` took and chose.

    offsets: int32 [S + 1], where the packed sequences begin and the last one ends (None: all tokens
    are one sequence); mask: bool [T], False for tokens that take no part, like those outside all
    sequences. topk_ids[T, k + n_shared]; ids outside [0, E) and the shared slots are not counted."""
    return BalanceLoss._make(S.balance_loss(logits, topk_ids, mode, logit_bias, n_shared, offsets, mask))


def balance_loss_backward(dlosses, logits, saved: BalanceLoss, k: int, mode: int = L.MOE_ROUTE_SOFTMAX,
                          logit_bias=None, offsets=None, mask=None, dlogits=None):
    """dlogits[T, E] from dlosses, fp32 [2] on the device (each loss's weight in the total, times any loss
    scale). Added to `dlogits` in place where that is given, as ``route_backward`` left it. k: the
    routed slots a token; the rest as for ``balance_loss``. Counts have no gradient."""
    return S.balance_loss_backward(dlosses, logits, saved.counts, saved.tokens, saved.totals, k, mode,
                                   logit_bias, offsets, mask, dlogits)
