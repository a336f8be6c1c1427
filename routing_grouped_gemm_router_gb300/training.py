"""The operators that train a sparse block, on tensors: checks of arguments, output and
workspace allocation (PyTorch's caching allocator, current stream) around the C entry points
of ``include/moe_train.h``, which says what each computes.

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

_DTYPES = {torch.bfloat16: L.MOE_BF16, torch.float32: L.MOE_F32}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _rows(name, t, shape, dtype=None):
    """A contiguous bf16 or fp32 CUDA tensor of `shape` (None: any extent)."""
    _need(isinstance(t, torch.Tensor), f"{name}: a tensor is needed")
    _need(t.dtype in _DTYPES if dtype is None else t.dtype == dtype,
          f"{name}: dtype {t.dtype}, expected {dtype or 'bfloat16 or float32'}")
    _need(t.dim() == len(shape) and all(a is None or a == b for a, b in zip(shape, t.shape)),
          f"{name}: shape {tuple(t.shape)}, expected {shape}")
    _need(t.is_contiguous(), f"{name}: has to be contiguous (strides {t.stride()})")
    _need(t.is_cuda, f"{name}: has to be on a CUDA device")
    return t


def _ints(name, t, shape):
    return _rows(name, t, shape, torch.int32)


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
    _ints("topk_ids", topk_ids, (None, None))
    T, k = topk_ids.shape
    P = buffer_rows(T, k, E)
    _need(P > 0 and E >= k, f"topk_ids: {T} tokens, {k} of {E} experts")
    ws_bytes = L.moe_align_workspace_size(T, k, E, L.MOE_TRAIN_BLOCK)
    blocks = P // L.MOE_TRAIN_BLOCK
    # one allocation: sorted_ids, then expert_ids, counts and the total, then scratch
    buf = torch.empty(P + blocks + E + 1 + (ws_bytes + 3) // 4, dtype=torch.int32,
                      device=topk_ids.device)
    sid, eid, counts, npp, ws = buf.split([P, blocks, E, 1, buf.numel() - P - blocks - E - 1])
    L.moe_align(topk_ids, T, k, E, L.MOE_TRAIN_BLOCK, sid, eid, npp, counts,
                ws if ws_bytes else None, ws_bytes)
    return SortedTokens(sid, eid, npp, counts)


def permute(x, topk_ids, sorted_ids, E: int):
    """(xs[rows, H], row_pos[T, k]): token rows copied to their slots' rows; -1 for dropped slots."""
    _rows("x", x, (None, None))
    T, H = x.shape
    _ints("topk_ids", topk_ids, (T, None))
    _ints("sorted_ids", sorted_ids, (None,))
    k, P = topk_ids.shape[1], sorted_ids.shape[0]
    xs = torch.empty(P, H, dtype=x.dtype, device=x.device)
    pos = torch.empty(T, k, dtype=torch.int32, device=x.device)
    L.moe_permute(x, topk_ids, sorted_ids, T, k, E, H, _DTYPES[x.dtype], P, xs, pos)
    return xs, pos


def permute_backward(dxs, row_pos):
    """dx[T, H]: the gradients of a token's rows summed over its slots."""
    _rows("dxs", dxs, (None, None))
    _ints("row_pos", row_pos, (None, None))
    (P, H), (T, k) = dxs.shape, row_pos.shape
    dx = torch.empty(T, H, dtype=dxs.dtype, device=dxs.device)
    L.moe_permute_backward(dxs, row_pos, T, k, H, _DTYPES[dxs.dtype], P, dx)
    return dx


def unpermute(ys, row_pos, topk_w):
    """out[T, H]: the rows of a token's slots, weighted and summed."""
    _rows("ys", ys, (None, None))
    _ints("row_pos", row_pos, (None, None))
    (P, H), (T, k) = ys.shape, row_pos.shape
    _rows("topk_w", topk_w, (T, k), torch.float32)
    out = torch.empty(T, H, dtype=ys.dtype, device=ys.device)
    L.moe_unpermute(ys, row_pos, topk_w, T, k, H, _DTYPES[ys.dtype], P, out)
    return out


def unpermute_backward(dout, ys, sorted_ids, row_pos, topk_w):
    """(dys[rows, H], dtopk_w[T, k]) of ``unpermute``."""
    _rows("ys", ys, (None, None))
    _ints("row_pos", row_pos, (None, None))
    (P, H), (T, k) = ys.shape, row_pos.shape
    _rows("dout", dout, (T, H), ys.dtype)
    _ints("sorted_ids", sorted_ids, (P,))
    _rows("topk_w", topk_w, (T, k), torch.float32)
    dys, dw = torch.empty_like(ys), torch.empty_like(topk_w)
    L.moe_unpermute_backward(dout, ys, sorted_ids, row_pos, topk_w, T, k, H, _DTYPES[ys.dtype],
                             P, dys, dw)
    return dys, dw


# -------------------------------------------------------------------------------- experts
def _experts_cfg(P, E, H, I, dtype):
    return L.moe_experts_t(P, E, H, I, _DTYPES[dtype])


def expert_up(xs, W13, counts):
    """(h13[rows, 2I], act[rows, I]): gate and up projections (fp32, kept for the backward pass) and
    silu(gate) * up of every expert's rows."""
    _rows("xs", xs, (None, None))
    P, H = xs.shape
    _rows("W13", W13, (None, None, H), xs.dtype)
    E, I2 = W13.shape[:2]
    _need(I2 % 2 == 0, f"W13: {I2} rows are no gate and up halves")
    _ints("counts", counts, (E,))
    h13 = torch.empty(P, I2, dtype=torch.float32, device=xs.device)
    act = torch.empty(P, I2 // 2, dtype=xs.dtype, device=xs.device)
    L.moe_expert_up(_experts_cfg(P, E, H, I2 // 2, xs.dtype), xs, W13, counts, h13, act)
    return h13, act


def expert_down(act, W2, counts):
    """ys[rows, H]: the down projection of every expert's rows, without the router weight."""
    _rows("act", act, (None, None))
    P, I = act.shape
    _rows("W2", W2, (None, None, I), act.dtype)
    E, H = W2.shape[:2]
    _ints("counts", counts, (E,))
    ys = torch.empty(P, H, dtype=act.dtype, device=act.device)
    L.moe_expert_down(_experts_cfg(P, E, H, I, act.dtype), act, W2, counts, ys)
    return ys


def expert_down_backward(dys, W2, h13, counts):
    """(dh13[rows, 2I], act[rows, I]): the gradient through the down projection and the SwiGLU, and
    the activations computed again for the gradient of W2."""
    _rows("dys", dys, (None, None))
    P, H = dys.shape
    _rows("W2", W2, (None, H, None), dys.dtype)
    E, I = W2.shape[0], W2.shape[2]
    _rows("h13", h13, (P, 2 * I), torch.float32)
    _ints("counts", counts, (E,))
    dh13 = torch.empty(P, 2 * I, dtype=dys.dtype, device=dys.device)
    act = torch.empty(P, I, dtype=dys.dtype, device=dys.device)
    L.moe_expert_down_backward(_experts_cfg(P, E, H, I, dys.dtype), dys, W2, h13, counts, dh13, act)
    return dh13, act


def expert_up_backward(dh13, W13, counts):
    """dxs[rows, H]: the gradient through the gate and up projections."""
    _rows("dh13", dh13, (None, None))
    P, I2 = dh13.shape
    _rows("W13", W13, (None, I2, None), dh13.dtype)
    _need(I2 % 2 == 0, f"dh13: {I2} columns are no gate and up halves")
    E, H = W13.shape[0], W13.shape[2]
    _ints("counts", counts, (E,))
    dxs = torch.empty(P, H, dtype=dh13.dtype, device=dh13.device)
    L.moe_expert_up_backward(_experts_cfg(P, E, H, I2 // 2, dh13.dtype), dh13, W13, counts, dxs)
    return dxs


def expert_weight_grad(dy, a, counts, out: Optional[torch.Tensor] = None,
                       out_dtype: Optional[torch.dtype] = None, accumulate: bool = False):
    """dW[E, M, N] = dy_e^T a_e over every expert's rows: W2's gradient from (dys, act), W13's from
    (dh13, xs). `out` (then its dtype counts) is overwritten, or added to with `accumulate`;
    otherwise a new tensor of out_dtype (default: dy's) is returned."""
    _rows("dy", dy, (None, None))
    P, M = dy.shape
    _rows("a", a, (P, None), dy.dtype)
    _ints("counts", counts, (None,))
    E, N = counts.shape[0], a.shape[1]
    if out is None:
        _need(not accumulate, "accumulate: needs the tensor to add to (out)")
        out = torch.empty(E, M, N, dtype=out_dtype or dy.dtype, device=dy.device)
    _rows("out", out, (E, M, N), out_dtype)
    L.moe_expert_weight_grad(P, E, M, N, _DTYPES[dy.dtype], _DTYPES[out.dtype], accumulate, dy, a,
                             counts, out)
    return out


# -------------------------------------------------------------------- norms around the block
def _gate_kind(gate, T, H, dtype):
    if gate is None:
        return L.MOE_GATE_NONE
    shape = tuple(gate.shape)
    if shape == (H,):
        _rows("gate", gate, (H,), torch.float32)
        return L.MOE_GATE_CHANNEL
    if shape == (T, 1):
        _rows("gate", gate, (T, 1), torch.float32)
        return L.MOE_GATE_TOKEN
    _rows("gate", gate, (T, H), dtype)
    return L.MOE_GATE_FULL


def _block_ws(cfg, device):
    n = L.moe_block_workspace_size(cfg)
    return torch.empty(n, dtype=torch.uint8, device=device), n


def block_norm(x, gamma, eps: float = 1e-6, offset: float = 0.0):
    """(h, rstd): x * rstd * (offset + gamma), rstd = (mean(x^2) + eps)^-1/2 of each row."""
    _rows("x", x, (None, None))
    T, H = x.shape
    _rows("gamma", gamma, (H,), torch.float32)
    h, rstd = torch.empty_like(x), torch.empty(T, dtype=torch.float32, device=x.device)
    L.moe_block_norm(L.moe_block_t(T, H, _DTYPES[x.dtype], 0, 1.0, offset, eps), x, gamma, h, rstd)
    return h, rstd


def block_norm_backward(dh, x, gamma, rstd, dres=None, offset: float = 0.0):
    """(dx, dgamma) of ``block_norm``; dres, the gradient that reaches x past the norm, is added."""
    _rows("x", x, (None, None))
    T, H = x.shape
    _rows("dh", dh, (T, H), x.dtype)
    _rows("gamma", gamma, (H,), torch.float32)
    _rows("rstd", rstd, (T,), torch.float32)
    if dres is not None:
        _rows("dres", dres, (T, H), x.dtype)
    cfg = L.moe_block_t(T, H, _DTYPES[x.dtype], 0, 1.0, offset, 0.0)
    ws, n = _block_ws(cfg, x.device)
    dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
    L.moe_block_norm_backward(cfg, dh, x, gamma, rstd, dres, dx, dgamma, ws, n)
    return dx, dgamma


class Joined(NamedTuple):
    out: torch.Tensor
    rstd_y: torch.Tensor
    h: Optional[torch.Tensor]         # the next block's normed input
    rstd_out: Optional[torch.Tensor]


def block_join(x, y, gamma, gate=None, scale: float = 1.0, gamma_next=None, eps: float = 1e-6,
               offset: float = 0.0) -> Joined:
    """out = x + scale * gate * norm(y; gamma), and h = norm(out; gamma_next) of the same pass.
    gate: None, fp32 [H] (a channel), fp32 [T, 1] (a token) or [T, H] of x's dtype."""
    _rows("x", x, (None, None))
    T, H = x.shape
    _rows("y", y, (T, H), x.dtype)
    _rows("gamma", gamma, (H,), torch.float32)
    kind = _gate_kind(gate, T, H, x.dtype)
    out, rstd_y = torch.empty_like(x), torch.empty(T, dtype=torch.float32, device=x.device)
    h = rstd_out = None
    if gamma_next is not None:
        _rows("gamma_next", gamma_next, (H,), torch.float32)
        h, rstd_out = torch.empty_like(x), torch.empty_like(rstd_y)
    L.moe_block_join(L.moe_block_t(T, H, _DTYPES[x.dtype], kind, scale, offset, eps), x, y, gamma,
                     gate, gamma_next, out, rstd_y, h, rstd_out)
    return Joined(out, rstd_y, h, rstd_out)


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
    _rows("y", y, (None, None))
    T, H = y.shape
    _rows("gamma", gamma, (H,), torch.float32)
    _rows("rstd_y", rstd_y, (T,), torch.float32)
    if dres is not None:
        _rows("dres", dres, (T, H), y.dtype)
    given = [t is not None for t in (dh, out, gamma_next, rstd_out)]
    _need(all(given) or not any(given), "dh, out, gamma_next and rstd_out are given together")
    _need(dres is not None or dh is not None, "dres or dh: a gradient is needed")
    dgn = None
    if dh is not None:
        _rows("dh", dh, (T, H), y.dtype)
        _rows("out", out, (T, H), y.dtype)
        _rows("gamma_next", gamma_next, (H,), torch.float32)
        _rows("rstd_out", rstd_out, (T,), torch.float32)
        dgn = torch.empty_like(gamma_next)
    kind = _gate_kind(gate, T, H, y.dtype)
    dgate = torch.empty_like(gate) if gate is not None else None
    cfg = L.moe_block_t(T, H, _DTYPES[y.dtype], kind, scale, offset, 0.0)
    ws, n = _block_ws(cfg, y.device)
    dx, dy, dg = torch.empty_like(y), torch.empty_like(y), torch.empty_like(gamma)
    L.moe_block_join_backward(cfg, dres, dh, out, y, gamma, gate, gamma_next, rstd_y, rstd_out, dx,
                              dy, dg, dgn, dgate, ws, n)
    return JoinGrads(dx, dy, dg, dgn, dgate)


# --------------------------------------------------------------------------------- router
def route_backward(logits, topk_ids, dtopk_w, mode: int = L.MOE_ROUTE_SOFTMAX,
                   renormalize: bool = True, scale: float = 1.0, logit_bias=None,
                   n_shared: int = 0):
    """dlogits[T, E] from the gradient of ``moe_route``'s topk_w, for the ids it chose."""
    _rows("logits", logits, (None, None), torch.float32)
    T, E = logits.shape
    _ints("topk_ids", topk_ids, (T, None))
    slots = topk_ids.shape[1]
    _rows("dtopk_w", dtopk_w, (T, slots), torch.float32)
    if logit_bias is not None:
        _rows("logit_bias", logit_bias, (E,), torch.float32)
    cfg = L.make_config(T, 8, 8, E, slots - n_shared, L.MOE_F32, mode, renormalize, scale,
                        logit_bias=logit_bias, n_shared=n_shared)
    dlogits = torch.empty_like(logits)
    L.moe_route_backward(cfg, logits, topk_ids, dtopk_w, dlogits)
    return dlogits
