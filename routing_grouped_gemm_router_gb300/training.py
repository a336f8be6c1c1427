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

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib as L

_C = L.lib()
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_DTYPES = {_BF16: L.MOE_BF16, _F32: L.MOE_F32}
_empty, _empty_like, _byref = torch.empty, torch.empty_like, ctypes.byref


# The checks run on every call of operators that take a few microseconds, so a good tensor
# passes in one expression and only a bad one is described.
def _refuse(name, t, shape, dtype):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if (t.dtype not in _DTYPES) if dtype is None else (t.dtype != dtype):
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype or 'bfloat16 or float32'}")
    if t.dim() != len(shape) or any(a is not None and a != b for a, b in zip(shape, t.shape)):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous (strides {t.stride()})")
    if not t.is_cuda:
        raise ValueError(f"{name}: has to be on a CUDA device")
    raise ValueError(f"{name}: is on {t.device}, not on the device of the other tensors")


def _first(name, t):
    """The first tensor of a call, bf16 or fp32 [a, b]: its two extents and device."""
    try:
        if t.dtype in _DTYPES and t.is_contiguous() and t.is_cuda:
            a, b = t.shape
            return a, b, t.get_device()
    except (AttributeError, ValueError):
        pass
    _refuse(name, t, (None, None), None)


def _like(name, t, shape, dtype, dev):
    """A further tensor: this very shape, type and device."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return
    except AttributeError:
        pass
    _refuse(name, t, shape, dtype)


def _any2(name, t, dtype, dev, rows=None):
    """A further tensor [rows or any, any] of this type: its two extents."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            a, b = t.shape
            if rows is None or a == rows:
                return a, b
    except (AttributeError, ValueError):
        pass
    _refuse(name, t, (rows, None), dtype)


def _weights(name, t, shape, dtype, dev):
    """Expert weights: three extents, those of `shape` that are not None given."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.dim() == 3 and \
                all(a is None or a == b for a, b in zip(shape, t.shape)):
            return t.shape
    except AttributeError:
        pass
    _refuse(name, t, shape, dtype)


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _done(fn, status):
    if status:
        raise L.MoeError(fn, status)


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
    dev = topk_ids.get_device() if isinstance(topk_ids, torch.Tensor) else -1
    T, k = _any2("topk_ids", topk_ids, _I32, dev)
    if dev < 0:
        _refuse("topk_ids", topk_ids, (None, None), _I32)
    P = buffer_rows(T, k, E)
    if P <= 0 or E < k:
        raise ValueError(f"topk_ids: {T} tokens, {k} of {E} experts")
    ws_bytes = L.moe_align_workspace_size(T, k, E, L.MOE_TRAIN_BLOCK)
    blocks, words = P // L.MOE_TRAIN_BLOCK, (ws_bytes + 3) // 4
    # one allocation: sorted_ids, then expert_ids, counts and the total, then scratch
    buf = _empty(P + blocks + E + 1 + words, dtype=_I32, device=topk_ids.device)
    sid, eid, counts, npp, ws = buf.split([P, blocks, E, 1, words])
    p = buf.data_ptr()
    _done("moe_align", _C.moe_align(
        topk_ids.data_ptr(), T, k, E, L.MOE_TRAIN_BLOCK, p, p + 4 * P, p + 4 * (P + blocks + E),
        p + 4 * (P + blocks), p + 4 * (P + blocks + E + 1) if words else None, ws_bytes,
        _stream(dev)))
    return SortedTokens(sid, eid, npp, counts)


def permute(x, topk_ids, sorted_ids, E: int):
    """(xs[rows, H], row_pos[T, k]): token rows copied to their slots' rows; -1 for dropped slots."""
    T, H, dev = _first("x", x)
    k = _any2("topk_ids", topk_ids, _I32, dev, T)[1]
    P = sorted_ids.shape[0]
    _like("sorted_ids", sorted_ids, (P,), _I32, dev)
    xs = _empty(P, H, dtype=x.dtype, device=x.device)
    pos = _empty_like(topk_ids)
    _done("moe_permute", _C.moe_permute(
        x.data_ptr(), topk_ids.data_ptr(), sorted_ids.data_ptr(), T, k, E, H, _DTYPES[x.dtype], P,
        xs.data_ptr(), pos.data_ptr(), _stream(dev)))
    return xs, pos


def permute_backward(dxs, row_pos):
    """dx[T, H]: the gradients of a token's rows summed over its slots."""
    P, H, dev = _first("dxs", dxs)
    T, k = _any2("row_pos", row_pos, _I32, dev)
    dx = _empty(T, H, dtype=dxs.dtype, device=dxs.device)
    _done("moe_permute_backward", _C.moe_permute_backward(
        dxs.data_ptr(), row_pos.data_ptr(), T, k, H, _DTYPES[dxs.dtype], P, dx.data_ptr(),
        _stream(dev)))
    return dx


def unpermute(ys, row_pos, topk_w):
    """out[T, H]: the rows of a token's slots, weighted and summed."""
    P, H, dev = _first("ys", ys)
    T, k = _any2("row_pos", row_pos, _I32, dev)
    _like("topk_w", topk_w, (T, k), _F32, dev)
    out = _empty(T, H, dtype=ys.dtype, device=ys.device)
    _done("moe_unpermute", _C.moe_unpermute(
        ys.data_ptr(), row_pos.data_ptr(), topk_w.data_ptr(), T, k, H, _DTYPES[ys.dtype], P,
        out.data_ptr(), _stream(dev)))
    return out


def unpermute_backward(dout, ys, sorted_ids, row_pos, topk_w):
    """(dys[rows, H], dtopk_w[T, k]) of ``unpermute``."""
    P, H, dev = _first("ys", ys)
    T, k = _any2("row_pos", row_pos, _I32, dev)
    _like("dout", dout, (T, H), ys.dtype, dev)
    _like("sorted_ids", sorted_ids, (P,), _I32, dev)
    _like("topk_w", topk_w, (T, k), _F32, dev)
    dys, dw = _empty_like(ys), _empty_like(topk_w)
    _done("moe_unpermute_backward", _C.moe_unpermute_backward(
        dout.data_ptr(), ys.data_ptr(), sorted_ids.data_ptr(), row_pos.data_ptr(),
        topk_w.data_ptr(), T, k, H, _DTYPES[ys.dtype], P, dys.data_ptr(), dw.data_ptr(),
        _stream(dev)))
    return dys, dw


# -------------------------------------------------------------------------------- experts
def _experts_cfg(P, E, H, I, dtype):
    return _byref(L.moe_experts_t(P, E, H, I, _DTYPES[dtype]))


def expert_up(xs, W13, counts):
    """(h13[rows, 2I], act[rows, I]): gate and up projections (fp32, kept for the backward pass) and
    silu(gate) * up of every expert's rows."""
    P, H, dev = _first("xs", xs)
    E, I2, _ = _weights("W13", W13, (None, None, H), xs.dtype, dev)
    if I2 % 2:
        raise ValueError(f"W13: {I2} rows are no gate and up halves")
    _like("counts", counts, (E,), _I32, dev)
    h13 = _empty(P, I2, dtype=_F32, device=xs.device)
    act = _empty(P, I2 // 2, dtype=xs.dtype, device=xs.device)
    _done("moe_expert_up", _C.moe_expert_up(
        _experts_cfg(P, E, H, I2 // 2, xs.dtype), xs.data_ptr(), W13.data_ptr(),
        counts.data_ptr(), h13.data_ptr(), act.data_ptr(), _stream(dev)))
    return h13, act


def expert_down(act, W2, counts):
    """ys[rows, H]: the down projection of every expert's rows, without the router weight."""
    P, I, dev = _first("act", act)
    E, H, _ = _weights("W2", W2, (None, None, I), act.dtype, dev)
    _like("counts", counts, (E,), _I32, dev)
    ys = _empty(P, H, dtype=act.dtype, device=act.device)
    _done("moe_expert_down", _C.moe_expert_down(
        _experts_cfg(P, E, H, I, act.dtype), act.data_ptr(), W2.data_ptr(), counts.data_ptr(),
        ys.data_ptr(), _stream(dev)))
    return ys


def expert_down_backward(dys, W2, h13, counts):
    """(dh13[rows, 2I], act[rows, I]): the gradient through the down projection and the SwiGLU, and
    the activations computed again for the gradient of W2."""
    P, H, dev = _first("dys", dys)
    E, _, I = _weights("W2", W2, (None, H, None), dys.dtype, dev)
    _like("h13", h13, (P, 2 * I), _F32, dev)
    _like("counts", counts, (E,), _I32, dev)
    dh13 = _empty(P, 2 * I, dtype=dys.dtype, device=dys.device)
    act = _empty(P, I, dtype=dys.dtype, device=dys.device)
    _done("moe_expert_down_backward", _C.moe_expert_down_backward(
        _experts_cfg(P, E, H, I, dys.dtype), dys.data_ptr(), W2.data_ptr(), h13.data_ptr(),
        counts.data_ptr(), dh13.data_ptr(), act.data_ptr(), _stream(dev)))
    return dh13, act


def expert_up_backward(dh13, W13, counts):
    """dxs[rows, H]: the gradient through the gate and up projections."""
    P, I2, dev = _first("dh13", dh13)
    E, _, H = _weights("W13", W13, (None, I2, None), dh13.dtype, dev)
    if I2 % 2:
        raise ValueError(f"dh13: {I2} columns are no gate and up halves")
    _like("counts", counts, (E,), _I32, dev)
    dxs = _empty(P, H, dtype=dh13.dtype, device=dh13.device)
    _done("moe_expert_up_backward", _C.moe_expert_up_backward(
        _experts_cfg(P, E, H, I2 // 2, dh13.dtype), dh13.data_ptr(), W13.data_ptr(),
        counts.data_ptr(), dxs.data_ptr(), _stream(dev)))
    return dxs


def expert_weight_grad(dy, a, counts, out: Optional[torch.Tensor] = None,
                       out_dtype: Optional[torch.dtype] = None, accumulate: bool = False):
    """dW[E, M, N] = dy_e^T a_e over every expert's rows: W2's gradient from (dys, act), W13's from
    (dh13, xs). `out` (then its dtype counts) is overwritten, or added to with `accumulate`;
    otherwise a new tensor of out_dtype (default: dy's) is returned."""
    P, M, dev = _first("dy", dy)
    N = _any2("a", a, dy.dtype, dev, P)[1]
    E = counts.numel()
    _like("counts", counts, (E,), _I32, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs the tensor to add to (out)")
        out = _empty(E, M, N, dtype=out_dtype or dy.dtype, device=dy.device)
    _like("out", out, (E, M, N), out_dtype or out.dtype, dev)
    if out.dtype not in _DTYPES:
        _refuse("out", out, (E, M, N), None)
    _done("moe_expert_weight_grad", _C.moe_expert_weight_grad(
        P, E, M, N, _DTYPES[dy.dtype], _DTYPES[out.dtype], int(bool(accumulate)), dy.data_ptr(),
        a.data_ptr(), counts.data_ptr(), out.data_ptr(), _stream(dev)))
    return out


# -------------------------------------------------------------------- norms around the block
def _gate_kind(gate, T, H, dtype, dev):
    if gate is None:
        return L.MOE_GATE_NONE
    if gate.shape == (H,):
        _like("gate", gate, (H,), _F32, dev)
        return L.MOE_GATE_CHANNEL
    if gate.shape == (T, 1):
        _like("gate", gate, (T, 1), _F32, dev)
        return L.MOE_GATE_TOKEN
    _like("gate", gate, (T, H), dtype, dev)
    return L.MOE_GATE_FULL


def _block_ws(cfg, device):
    n = ctypes.c_size_t(0)
    _done("moe_block_workspace_size", _C.moe_block_workspace_size(_byref(cfg), _byref(n)))
    return _empty(n.value, dtype=torch.uint8, device=device), n.value


def block_norm(x, gamma, eps: float = 1e-6, offset: float = 0.0):
    """(h, rstd): x * rstd * (offset + gamma), rstd = (mean(x^2) + eps)^-1/2 of each row."""
    T, H, dev = _first("x", x)
    _like("gamma", gamma, (H,), _F32, dev)
    h, rstd = _empty_like(x), _empty(T, dtype=_F32, device=x.device)
    cfg = L.moe_block_t(T, H, _DTYPES[x.dtype], 0, 1.0, offset, eps)
    _done("moe_block_norm", _C.moe_block_norm(
        _byref(cfg), x.data_ptr(), gamma.data_ptr(), h.data_ptr(), rstd.data_ptr(), _stream(dev)))
    return h, rstd


def block_norm_backward(dh, x, gamma, rstd, dres=None, offset: float = 0.0):
    """(dx, dgamma) of ``block_norm``; dres, the gradient that reaches x past the norm, is added."""
    T, H, dev = _first("x", x)
    _like("dh", dh, (T, H), x.dtype, dev)
    _like("gamma", gamma, (H,), _F32, dev)
    _like("rstd", rstd, (T,), _F32, dev)
    if dres is not None:
        _like("dres", dres, (T, H), x.dtype, dev)
    cfg = L.moe_block_t(T, H, _DTYPES[x.dtype], 0, 1.0, offset, 0.0)
    ws, n = _block_ws(cfg, x.device)
    dx, dgamma = _empty_like(x), _empty_like(gamma)
    _done("moe_block_norm_backward", _C.moe_block_norm_backward(
        _byref(cfg), dh.data_ptr(), x.data_ptr(), gamma.data_ptr(), rstd.data_ptr(),
        dres.data_ptr() if dres is not None else None, dx.data_ptr(), dgamma.data_ptr(),
        ws.data_ptr(), n, _stream(dev)))
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
    T, H, dev = _first("x", x)
    _like("y", y, (T, H), x.dtype, dev)
    _like("gamma", gamma, (H,), _F32, dev)
    kind = _gate_kind(gate, T, H, x.dtype, dev)
    out, rstd_y = _empty_like(x), _empty(T, dtype=_F32, device=x.device)
    h = rstd_out = None
    if gamma_next is not None:
        _like("gamma_next", gamma_next, (H,), _F32, dev)
        h, rstd_out = _empty_like(x), _empty_like(rstd_y)
    cfg = L.moe_block_t(T, H, _DTYPES[x.dtype], kind, scale, offset, eps)
    nxt = h is not None
    _done("moe_block_join", _C.moe_block_join(
        _byref(cfg), x.data_ptr(), y.data_ptr(), gamma.data_ptr(), gate.data_ptr() if kind else None,
        gamma_next.data_ptr() if nxt else None, out.data_ptr(), rstd_y.data_ptr(),
        h.data_ptr() if nxt else None, rstd_out.data_ptr() if nxt else None, _stream(dev)))
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
    T, H, dev = _first("y", y)
    _like("gamma", gamma, (H,), _F32, dev)
    _like("rstd_y", rstd_y, (T,), _F32, dev)
    if dres is not None:
        _like("dres", dres, (T, H), y.dtype, dev)
    nxt = dh is not None
    if any((t is not None) != nxt for t in (out, gamma_next, rstd_out)):
        raise ValueError("dh, out, gamma_next and rstd_out are given together")
    if dres is None and not nxt:
        raise ValueError("dres or dh: a gradient is needed")
    dgn = None
    if nxt:
        _like("dh", dh, (T, H), y.dtype, dev)
        _like("out", out, (T, H), y.dtype, dev)
        _like("gamma_next", gamma_next, (H,), _F32, dev)
        _like("rstd_out", rstd_out, (T,), _F32, dev)
        dgn = _empty_like(gamma_next)
    kind = _gate_kind(gate, T, H, y.dtype, dev)
    dgate = _empty_like(gate) if kind else None
    cfg = L.moe_block_t(T, H, _DTYPES[y.dtype], kind, scale, offset, 0.0)
    ws, n = _block_ws(cfg, y.device)
    dx, dy, dg = _empty_like(y), _empty_like(y), _empty_like(gamma)
    _done("moe_block_join_backward", _C.moe_block_join_backward(
        _byref(cfg), dres.data_ptr() if dres is not None else None, dh.data_ptr() if nxt else None,
        out.data_ptr() if nxt else None, y.data_ptr(), gamma.data_ptr(),
        gate.data_ptr() if kind else None, gamma_next.data_ptr() if nxt else None,
        rstd_y.data_ptr(), rstd_out.data_ptr() if nxt else None, dx.data_ptr(), dy.data_ptr(),
        dg.data_ptr(), dgn.data_ptr() if nxt else None, dgate.data_ptr() if kind else None,
        ws.data_ptr(), n, _stream(dev)))
    return JoinGrads(dx, dy, dg, dgn, dgate)


# --------------------------------------------------------------------------------- router
def route_backward(logits, topk_ids, dtopk_w, mode: int = L.MOE_ROUTE_SOFTMAX,
                   renormalize: bool = True, scale: float = 1.0, logit_bias=None,
                   n_shared: int = 0):
    """dlogits[T, E] from the gradient of ``moe_route``'s topk_w, for the ids it chose."""
    dev = logits.get_device() if isinstance(logits, torch.Tensor) else -1
    T, E = _any2("logits", logits, _F32, dev)
    if dev < 0:
        _refuse("logits", logits, (None, None), _F32)
    slots = _any2("topk_ids", topk_ids, _I32, dev, T)[1]
    _like("dtopk_w", dtopk_w, (T, slots), _F32, dev)
    if logit_bias is not None:
        _like("logit_bias", logit_bias, (E,), _F32, dev)
    cfg = L.moe_config_t(T=T, E=E, k=slots - n_shared, mode=mode, renormalize=int(bool(renormalize)),
                         scale=scale, n_shared=n_shared,
                         logit_bias=logit_bias.data_ptr() if logit_bias is not None else None)
    dlogits = _empty_like(logits)
    _done("moe_route_backward", _C.moe_route_backward(
        _byref(cfg), logits.data_ptr(), topk_ids.data_ptr(), dtopk_w.data_ptr(),
        dlogits.data_ptr(), _stream(dev)))
    return dlogits
