"""Torch-tensor wrapper of moe_adapters_add: low-rank adapters of many requests beside a shared projection.

The rows are grouped by adapter with moe_align over the adapters in the place of experts:

    plan = moe_align(adapter_ids.view(-1, 1), 0, n_adapters, block_m)      # -1: no adapter; once a step
    y = moe_w8a8_linear(q, qs, W, Ws)                                      # the projection that all share
    moe_adapters_add(y, x, A, B, plan, block_m, scales, out=y)             # y[m] += scale * B[a] (A[a] x[m])

block_m: the least of 16, 32 and 64 that holds an adapter's mean number of rows, 64 above.
"""
from __future__ import annotations

import ctypes as C
import functools
from typing import Optional

import torch

from . import _lib as L
from .experts import _BF16, _F32, _I32, _call, _check, _check_align, _ld, _live_ptr

_changed = torch._C._increment_version   # (torch.autograd.graph's function without its own checks: 0.3 us, not 0.7)


@functools.lru_cache(maxsize=256)
def adapters_workspace(numel: int, n_adapters: int, rank: int, K: int, block_m: int) -> int:
    """float32 values of moe_adapters_add's workspace for numel rows."""
    n = C.c_int64()
    L.check(L.lib().moe_adapters_workspace(numel, n_adapters, rank, K, block_m, C.byref(n)), "moe_adapters_workspace")
    return n.value


def moe_adapters_add(base: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, align, block_m: int,
                     scales: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None, top_k: int = 1,
                     out: Optional[torch.Tensor] = None, work: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[m] = base[m] + scales[a] * B[a] (A[a] x[m // top_k]) for the rows m of adapter a, base[m] for rows
    without one: base bf16 [numel, N], x bf16 [numel // top_k, K], A bf16 [n, r, K], B bf16 [n, N, r], scales
    float32 [n] (1 without), ranks int32 [n] (adapters of fewer than r ranks: what stands behind is not used).

    `align` is what moe_align returns for the rows' adapter ids [numel, 1] (expert_start 0, n_local n) with the same
    block_m.  `out`: base itself, or memory apart from it (allocated when not given); it may be x or lie over it.
    `work`: float32 workspace of adapters_workspace(numel, n, r, K, block_m) values (allocated when not given).

    For serving: the result has no gradient.  (Where autograd has kept an `out` from before, its backward pass refuses it
    as changed in place.)"""
    _check(base, "base", _BF16, rows=True)
    dev, (numel, N) = base.device, base.shape
    _check(x, "x", _BF16, dev=dev, rows=True)
    K = x.shape[1]
    if A.dim() != 3 or A.shape[2] != K:
        raise ValueError(f"A {tuple(A.shape)} must be [n, r, K] with the {K} columns of x")
    n, r, _ = A.shape
    _check(A, "A", _BF16, dev=dev)
    _check(B, "B", _BF16, (n, N, r), dev)
    if top_k < 1 or x.shape[0] * top_k != numel:
        raise ValueError(f"x has {x.shape[0]} rows for {numel} rows of base and top_k={top_k}")
    if scales is not None:
        _check(scales, "scales", _F32, (n,), dev)
    if ranks is not None:
        _check(ranks, "ranks", _I32, (n,), dev)
    sorted_ids, block_ids, padded, local = align
    _check_align(sorted_ids, block_ids, padded, numel, n, block_m, dev)
    live = _live_ptr(local, numel, dev)
    if out is None:
        out = torch.empty((numel, N), dtype=torch.bfloat16, device=dev)
    else:
        if out is not base:
            _check(out, "out", _BF16, (numel, N), dev, rows=True)
        if not out.is_inference():
            _changed((out,))
    if work is None:
        work = torch.empty(adapters_workspace(numel, n, r, K, block_m), dtype=torch.float32, device=dev)
    else:
        _check(work, "work", _F32, dev=dev)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call(dev, "moe_adapters_add", base.data_ptr(), _ld(base), x.data_ptr(), x.shape[0], _ld(x), A.data_ptr(), B.data_ptr(),
          p(scales), p(ranks), n, r, N, K, out.data_ptr(), _ld(out), sorted_ids.data_ptr(), block_ids.data_ptr(),
          padded.data_ptr(), live, numel, top_k, block_m, work.data_ptr(), work.numel())
    return out
