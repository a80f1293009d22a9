"""Torch-tensor wrappers of the experts' two ends: the router with its counts and balance loss, and the
gradients of the weighted combine.  One function for each C entry point, with the same name, and the
differentiable forms moe_experts_router and moe_experts_combine.

Tensors are checked for device, type and shape, outputs allocated with torch when not given, and
every computation runs in libmoe_w4a16 on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes as C
import functools
from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .experts import _BF16, _F32, _I32, _call, _check, _ld

_LOGITS = (torch.bfloat16, torch.float32)
_GRAD_TOKENS, _GRAD_NORM_COLUMNS = 1 << 24, 12288   # moe_combine_grad's limits


class RouterStats(NamedTuple):
    """Statistics of a batch: counts int32 [E], means float32 [E], balance float32 [1], tokens int32 [1]."""
    counts: torch.Tensor
    means: torch.Tensor
    balance: torch.Tensor
    tokens: torch.Tensor


class Routing(NamedTuple):
    """What moe_experts_router returns: ids int32 [M, k] and weights float32 [M, k] of the choices, counts
    int32 [E], means float32 [E] of the probabilities over the batch, and the balance loss, a float32 scalar."""
    ids: torch.Tensor
    weights: torch.Tensor
    counts: torch.Tensor
    means: torch.Tensor
    balance: torch.Tensor


@functools.lru_cache(maxsize=256)
def router_workspace(M: int, E: int) -> int:
    """Bytes of the workspace of moe_router's statistics."""
    n = C.c_int64()
    L.check(L.lib().moe_router_workspace(M, E, C.byref(n)), "moe_router_workspace")
    return n.value


def _score(score: str) -> int:
    kind = L.SCORE.get(score)
    if kind is None:
        raise ValueError(f"unknown score {score!r}")
    return kind


def _check_logits(logits, top_k, bias, live) -> None:
    _check(logits, "logits", _LOGITS, rows=True)
    M, E = logits.shape
    if bias is not None:
        _check(bias, "bias", _F32, (E,), logits.device)
    if live is not None:
        _check(live, "live", _I32, (M,), logits.device)


def _router(logits, top_k, kind, bias, live, renormalise, scale, ids, weights, stats, work) -> None:
    M, E = logits.shape
    _call(logits.device, "moe_router", logits.data_ptr(), logits.dtype is torch.float32, _ld(logits), M, E,
          None if bias is None else bias.data_ptr(), None if live is None else live.data_ptr(), kind, top_k, renormalise,
          scale, ids.data_ptr(), weights.data_ptr(), *((None,) * 4 if stats is None else [t.data_ptr() for t in stats]),
          None if work is None else work.data_ptr(), 0 if work is None else work.numel() * work.element_size())


def _new_outputs(M, E, top_k, dev):
    return (torch.empty((M, top_k), dtype=torch.int32, device=dev),
            torch.empty((M, top_k), dtype=torch.float32, device=dev))


def _new_stats(E, dev, balance=(1,)) -> RouterStats:
    return RouterStats(torch.empty(E, dtype=torch.int32, device=dev), torch.empty(E, dtype=torch.float32, device=dev),
                       torch.empty(balance, dtype=torch.float32, device=dev), torch.empty(1, dtype=torch.int32, device=dev))


def moe_router(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
               renormalise: bool = False, scale: float = 1.0, live: Optional[torch.Tensor] = None, out=None,
               stats=False, work: Optional[torch.Tensor] = None):
    """logits [M, E] (bf16 or float32) -> (topk_ids int32 [M, top_k], topk_weights float32 [M, top_k]): the
    experts of the largest logits -- with `bias` (float32 [E]) of the largest score + bias, the score being a
    softmax or a sigmoid -- and their scores, divided by their sum with `renormalise`, times `scale`.  Ties go to
    the lower index; -inf logits are never chosen, and choices left over have id -1 and weight 0.  `live` (int32
    [M]): tokens with a negative entry (padding) get ids -1 and weights 0.

    `stats`: True, or a RouterStats to write, and the result is (ids, weights, RouterStats): the experts' counts,
    their mean probabilities, the balance loss and the number of live tokens.  `work`: uint8 workspace of
    router_workspace(M, E) bytes for them (allocated when not given)."""
    kind = _score(score)
    _check_logits(logits, top_k, bias, live)
    (M, E), dev = logits.shape, logits.device
    if out is None:
        out = _new_outputs(M, E, max(top_k, 0), dev)
    ids, weights = out
    _check(ids, "topk_ids", _I32, (M, top_k), dev)
    _check(weights, "topk_weights", _F32, (M, top_k), dev)
    if not stats:
        _router(logits, top_k, kind, bias, live, renormalise, scale, ids, weights, None, None)
        return ids, weights
    if stats is True:
        stats = _new_stats(E, dev)
    else:
        stats = RouterStats(*stats)
        for t, name, dtypes, n in zip(stats, RouterStats._fields, (_I32, _F32, _F32, _I32), (E, E, 1, 1)):
            _check(t, name, dtypes, (n,), dev)
    if work is None:
        work = torch.empty(router_workspace(M, E), dtype=torch.uint8, device=dev)
    else:
        _check(work, "work", (torch.uint8,), dev=dev)
    _router(logits, top_k, kind, bias, live, renormalise, scale, ids, weights, stats, work)
    return ids, weights, stats


def _router_grad(logits, live, kind, top_k, renormalise, scale, ids, d_weights, counts, tokens, d_means, d_balance,
                 out) -> None:
    M, E = logits.shape
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call(logits.device, "moe_router_grad", logits.data_ptr(), logits.dtype is torch.float32, _ld(logits), M, E, p(live),
          kind, top_k, renormalise, scale, p(ids), p(d_weights), p(counts), p(tokens), p(d_means), p(d_balance),
          out.data_ptr(), _ld(out))


def moe_router_grad(logits: torch.Tensor, topk_ids: torch.Tensor, d_weights: Optional[torch.Tensor] = None,
                    score: str = "softmax", renormalise: bool = False, scale: float = 1.0,
                    live: Optional[torch.Tensor] = None, stats=None, d_means: Optional[torch.Tensor] = None,
                    d_balance: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of moe_router's weights (d_weights float32 [M, top_k]) and, from the `stats` it returned, of the
    means (d_means float32 [E]) and the balance loss (d_balance, one float32) with respect to the logits, in their
    type."""
    kind = _score(score)
    _check_logits(logits, 0, None, live)
    (M, E), dev = logits.shape, logits.device
    _check(topk_ids, "topk_ids", _I32, dev=dev)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != M:
        raise ValueError(f"topk_ids must be [{M}, top_k], got {tuple(topk_ids.shape)}")
    if d_weights is not None:
        _check(d_weights, "d_weights", _F32, tuple(topk_ids.shape), dev)
    if d_means is not None:
        _check(d_means, "d_means", _F32, (E,), dev)
    if d_balance is not None:
        _check(d_balance, "d_balance", _F32, dev=dev)
        if d_balance.numel() != 1:
            raise ValueError("d_balance must be one value")
    counts = tokens = None
    if d_means is not None or d_balance is not None:
        if stats is None:
            raise ValueError("d_means and d_balance need the router's stats")
        counts, _, _, tokens = stats
        _check(counts, "counts", _I32, (E,), dev)
        _check(tokens, "tokens", _I32, (1,), dev)
    if out is None:
        out = torch.empty((M, E), dtype=logits.dtype, device=dev)
    else:
        _check(out, "out", (logits.dtype,), (M, E), dev, rows=True)
    _router_grad(logits, live, kind, topk_ids.shape[1], renormalise, scale, topk_ids, d_weights, counts, tokens, d_means,
                 d_balance, out)
    return out


def _once(backward):
    """once_differentiable, without its time (5 us a call) where no second derivative can be asked for."""
    guarded = torch.autograd.function.once_differentiable(backward)

    @functools.wraps(backward)
    def call(ctx, *grads):
        return guarded(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return call


class _ExpertsRouter(torch.autograd.Function):
    # (`aside` takes the outputs without a gradient: each output of the function costs the graph's bookkeeping 5 us)
    @staticmethod
    def forward(ctx, logits, bias, live, top_k, kind, renormalise, scale, means_grad, aside):
        (M, E), dev = logits.shape, logits.device
        ids, weights = _new_outputs(M, E, top_k, dev)
        # (the loss of no dimension from the start: a view among several outputs could not be changed in place)
        counts, means, balance, tokens = stats = _new_stats(E, dev, ())
        work = torch.empty(router_workspace(M, E), dtype=torch.uint8, device=dev)
        _router(logits, top_k, kind, bias, live, renormalise, scale, ids, weights, stats, work)
        ctx.save_for_backward(logits, live, ids, counts, tokens)
        ctx.how = (kind, top_k, renormalise, scale)
        ctx.set_materialize_grads(False)
        aside += (ids, counts, means)
        return (weights, balance, means) if means_grad else (weights, balance)

    @staticmethod
    @_once
    def backward(ctx, d_weights, d_balance, d_means=None):
        logits, live, ids, counts, tokens = ctx.saved_tensors
        kind, top_k, renormalise, scale = ctx.how
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        if d_weights is not None and not d_weights.is_contiguous():   # (gradients may arrive broadcast)
            d_weights = d_weights.contiguous()
        if d_means is not None:
            d_means = d_means.contiguous()
        _router_grad(logits, live, kind, top_k, renormalise, scale, ids, d_weights, counts, tokens, d_means, d_balance, out)
        return out, None, None, None, None, None, None, None, None


def moe_experts_router(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                       renormalise: bool = False, scale: float = 1.0, live: Optional[torch.Tensor] = None,
                       means_grad: bool = False) -> Routing:
    """Differentiable moe_router with the batch's statistics: Routing(ids, weights, counts, means, balance).

    The gradients of weights and balance, and with `means_grad` of means, reach the logits in one pass; they have the
    logits' type and are once differentiable.  The choice, the counts and the selection bias have no gradient.  balance is
    E * sum_e (counts_e / sum counts) * means_e; for counts that are summed over several ranks' batches form the same
    sum from `means` (the ranks' mean of it is the loss of the whole batch when they hold equally many tokens).

    logits, live, ids and counts (for the gradient of balance and means alone) are read again in the backward pass: write
    over copies of them.  Forward and backward can be captured into a graph; as with any autograd work, hold no graph of
    an eager call of the same leaves while capturing."""
    kind = _score(score)
    _check_logits(logits, top_k, bias, live)
    if not 1 <= top_k <= logits.shape[1]:
        raise ValueError(f"top_k={top_k} of {logits.shape[1]} experts")
    aside = []
    out = _ExpertsRouter.apply(logits, bias, live, top_k, kind, renormalise, scale, means_grad, aside)
    ids, counts, means = aside
    return Routing(ids, out[0], counts, out[2] if means_grad else means, out[1])


@functools.lru_cache(maxsize=256)
def combine_grad_workspace(M: int, H: int) -> int:
    """float32 values of the workspace of moe_combine_grad's norm weight gradient."""
    n = C.c_int64()
    L.check(L.lib().moe_combine_grad_workspace(M, H, C.byref(n)), "moe_combine_grad_workspace")
    return n.value


def _combine_grad(y, weights, local, norm_w, eps, rsf, d_out, dy, d_weights, d_norm, work) -> None:
    M, k = weights.shape
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call(y.device, "moe_combine_grad", y.data_ptr(), weights.data_ptr(), local.data_ptr(), p(norm_w), eps, rsf, M, k,
          y.shape[1], d_out.data_ptr(), _ld(d_out), p(dy), p(d_weights), p(d_norm), p(work),
          0 if work is None else work.numel())


def _check_combine(y, topk_weights, slot_local_ids, norm_w) -> None:
    _check(y, "y", _BF16)
    _check(topk_weights, "topk_weights", _F32, dev=y.device)
    _check(slot_local_ids, "slot_local_ids", _I32, dev=y.device)
    if topk_weights.dim() != 2 or y.dim() != 2 or y.shape[0] != topk_weights.numel():
        raise ValueError(f"y {tuple(y.shape)} must have a row for each of the topk_weights {tuple(topk_weights.shape)}")
    if slot_local_ids.numel() != y.shape[0]:
        raise ValueError(f"slot_local_ids holds {slot_local_ids.numel()} ids for {y.shape[0]} slots")
    if norm_w is not None:
        _check(norm_w, "norm_w", _BF16, (y.shape[1],), y.device)


def moe_combine_grad(y: torch.Tensor, topk_weights: torch.Tensor, slot_local_ids: torch.Tensor, d_out: torch.Tensor,
                     norm_w: Optional[torch.Tensor] = None, eps: float = 1e-8, routed_scaling_factor: float = 1.0,
                     out=None, work: Optional[torch.Tensor] = None):
    """Gradients of moe_combine from d_out bf16 [M, H]: (dy bf16 [M * k, H], zero in rows of dead slots, d_weights
    float32 [M, k], d_norm_w bf16 [H] or None).  `out`: the three to write, None among them for a gradient that is
    not needed.  `work`: float32 workspace of combine_grad_workspace(M, H) values for d_norm_w (allocated when not
    given)."""
    _check_combine(y, topk_weights, slot_local_ids, norm_w)
    (M, k), H, dev = topk_weights.shape, y.shape[1], y.device
    _check(d_out, "d_out", _BF16, (M, H), dev, rows=True)
    if out is None:
        out = (torch.empty_like(y), torch.empty((M, k), dtype=torch.float32, device=dev),
               None if norm_w is None else torch.empty_like(norm_w))
    dy, d_weights, d_norm = out
    for t, name, dtypes, shape in ((dy, "dy", _BF16, (M * k, H)), (d_weights, "d_weights", _F32, (M, k)),
                                   (d_norm, "d_norm_w", _BF16, (H,))):
        if t is not None:
            _check(t, name, dtypes, shape, dev)
    if d_norm is not None:
        if work is None:
            work = torch.empty(combine_grad_workspace(M, H), dtype=torch.float32, device=dev)
        else:
            _check(work, "work", _F32, dev=dev)
    _combine_grad(y, topk_weights, slot_local_ids, norm_w, eps, routed_scaling_factor, d_out, dy, d_weights, d_norm, work)
    return dy, d_weights, d_norm


class _ExpertsCombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, norm_w, local, eps, rsf):
        (M, k), H = weights.shape, y.shape[1]
        out = torch.empty((M, H), dtype=torch.bfloat16, device=y.device)
        _call(y.device, "moe_combine", y.data_ptr(), weights.data_ptr(), local.data_ptr(),
              None if norm_w is None else norm_w.data_ptr(), eps, rsf, M, k, H, out.data_ptr())
        ctx.save_for_backward(y, weights, norm_w, local)
        ctx.how = (eps, rsf)
        return out

    @staticmethod
    @_once
    def backward(ctx, grad):
        y, weights, norm_w, local = ctx.saved_tensors
        # (a gradient may arrive broadcast or transposed, or with rows that 16-byte loads cannot take)
        if grad.stride(-1) != 1 or grad.stride(0) % 8 or grad.stride(0) < grad.shape[1] or grad.data_ptr() % 16:
            grad = grad.clone(memory_format=torch.contiguous_format)
        needs = ctx.needs_input_grad
        dy = torch.empty_like(y) if needs[0] else None
        dw = torch.empty_like(weights) if needs[1] else None
        dn = work = None
        if needs[2]:
            dn = torch.empty_like(norm_w)
            work = torch.empty(combine_grad_workspace(weights.shape[0], y.shape[1]), dtype=torch.float32, device=y.device)
        if dy is not None or dw is not None or dn is not None:
            _combine_grad(y, weights, local, norm_w, *ctx.how, grad, dy, dw, dn, work)
        return dy, dw, dn, None, None, None


def moe_experts_combine(y: torch.Tensor, topk_weights: torch.Tensor, slot_local_ids: torch.Tensor,
                        norm_w: Optional[torch.Tensor] = None, eps: float = 1e-8,
                        routed_scaling_factor: float = 1.0) -> torch.Tensor:
    """Differentiable moe_combine: out bf16 [M, H] from the slots' rows y bf16 [M * k, H] and the weights
    float32 [M, k] (the router's), optionally after the post-expert RMSNorm of weight norm_w bf16 [H] (the weight
    itself, moe_norm_weight's 1 + w).  Gradients flow to y, topk_weights and norm_w; they are once differentiable
    and zero for dead slots (slot_local_ids < 0).  With a gradient M is less than 2^24 tokens, and H at most 12288 columns
    for norm_w's.  All four tensors are read again in the backward pass: write over copies of them (what kernels write,
    a reused align's outputs among it, autograd does not see).

    Forward and backward can be captured into a graph; as with any autograd work, hold no graph of an eager call of
    the same leaves while capturing."""
    _check_combine(y, topk_weights, slot_local_ids, norm_w)
    M, H = topk_weights.shape[0], y.shape[1]
    if (M >= _GRAD_TOKENS or H > _GRAD_NORM_COLUMNS) and torch.is_grad_enabled():
        # (what the backward pass would refuse is refused before the forward one)
        d_norm = norm_w is not None and norm_w.requires_grad
        if M >= _GRAD_TOKENS and (y.requires_grad or topk_weights.requires_grad or d_norm):
            raise ValueError(f"{M} tokens: moe_combine_grad takes less than 2^24")
        if H > _GRAD_NORM_COLUMNS and d_norm:
            raise ValueError(f"norm_w of {H} columns: moe_combine_grad gives the gradient of at most {_GRAD_NORM_COLUMNS}")
    return _ExpertsCombine.apply(y, topk_weights, norm_w, slot_local_ids, eps, routed_scaling_factor)
