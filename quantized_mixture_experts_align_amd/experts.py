"""Torch-tensor wrappers of the experts with 8-bit and bf16 weights: one function for each C entry
point, with the same name, and moe_experts_linear, the differentiable form of moe_bf16_gemm.

Tensors are checked for device, type and shape, outputs allocated with torch when not given, and
every computation runs in libmoe_w4a16 on the current stream of the tensors' device.

block_m of the align: the least of 16, 32, 64 and 128 that holds a local expert's mean number of slots,
128 above.  expected_slots: on a slice of the experts tokens * top_k * n_local / n_experts.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L

GROUP = 128           # columns that share an activation scale, rows and columns of a weight block
_F8 = (torch.float8_e4m3fn, torch.uint8)


_entry = {}           # C entry points, looked up once
_raw_stream = torch._C._cuda_getCurrentRawStream   # (a stream's handle without a Stream object: 0.1 us, not 2.6)


def _call(dev: torch.device, name: str, *args) -> None:
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(L.lib(), name)
    index = dev.index
    if index == torch.cuda.current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(index))
    if rc:
        L.check(rc, name)


def _check(t: torch.Tensor, name: str, dtypes, shape=None, dev: Optional[torch.device] = None,
           rows: bool = False) -> None:
    """A device tensor of one of `dtypes` and of `shape`, contiguous (rows: a matrix whose rows are)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if rows:
        if t.dim() != 2 or (t.numel() and ((t.shape[1] > 1 and t.stride(1) != 1) or
                                           (t.shape[0] > 1 and t.stride(0) < t.shape[1]))):
            raise ValueError(f"{name} must be a matrix with contiguous, non-overlapping rows")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ld(t: torch.Tensor) -> int:
    """Values between rows (a single row's stride means nothing)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)


def _capacity(numel: int, E: int, block_m: int):
    """moe_align_capacity's slots and blocks (the entry points check the arguments themselves)."""
    if block_m < 1 or numel < 0:
        raise ValueError(f"numel={numel} block_m={block_m}")
    blocks = -(-(numel + min(E, numel) * (block_m - 1)) // block_m)
    return blocks * block_m, blocks


def _check_align(sorted_token_ids, expert_ids, num_tokens_post_padded, numel: int, E: int, block_m: int, dev) -> None:
    for t, name in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                    (num_tokens_post_padded, "num_tokens_post_padded")):
        _check(t, name, _I32, dev=dev)
    s_len, b_len = _capacity(numel, E, block_m)
    if sorted_token_ids.numel() < s_len or expert_ids.numel() < b_len or num_tokens_post_padded.numel() < 1:
        raise ValueError(f"the align's outputs hold {sorted_token_ids.numel()} slots and {expert_ids.numel()} blocks; "
                         f"{numel} slots on {E} experts in blocks of {block_m} need {s_len} and {b_len}")


def _quant_out(R: int, K: int, dev, out):
    if out is None:
        return (torch.empty((R, K), dtype=torch.float8_e4m3fn, device=dev),
                torch.empty((R, -(-K // GROUP)), dtype=torch.float32, device=dev))
    codes, scales = out
    _check(codes, "codes", _F8, (R, K), dev, rows=True)
    _check(scales, "scales", _F32, (R, -(-K // GROUP)), dev, rows=True)
    return codes, scales


def _live_ptr(slot_local_ids: Optional[torch.Tensor], R: int, dev) -> Optional[int]:
    if slot_local_ids is None:
        return None
    _check(slot_local_ids, "slot_local_ids", _I32, dev=dev)
    if slot_local_ids.numel() != R:
        raise ValueError(f"slot_local_ids holds {slot_local_ids.numel()} ids for {R} rows")
    return slot_local_ids.data_ptr()


def moe_fp8_quant(x: torch.Tensor, slot_local_ids: Optional[torch.Tensor] = None, out=None):
    """x bf16 [R, K] -> (codes float8_e4m3fn [R, K], scales fp32 [R, ceil(K/128)]): for each row and
    128 columns scale = max|x| / 448 and code = e4m3(x / scale).  Rows with slot_local_ids < 0 are
    neither read nor written.  `out`: the pair to write (codes may be uint8)."""
    _check(x, "x", _BF16, rows=True)
    R, K = x.shape
    codes, scales = _quant_out(R, K, x.device, out)
    _call(x.device, "moe_fp8_quant", x.data_ptr(), _ld(x), R, K, _live_ptr(slot_local_ids, R, x.device),
          codes.data_ptr(), _ld(codes), scales.data_ptr(), _ld(scales))
    return codes, scales


def moe_act_fp8_quant(kind: str, h: torch.Tensor, I: int, slot_local_ids: Optional[torch.Tensor] = None,
                      alpha: float = 1.702, limit: float = float("inf"), out=None):
    """moe_act and moe_fp8_quant in one pass: h bf16 [R, 2I] (gate, up; [R, I] for relu2) -> the
    activation's (codes [R, I], scales [R, ceil(I/128)]), quantised from fp32."""
    if kind not in L.ACT:
        raise ValueError(f"unknown activation {kind!r}")
    _check(h, "h", _BF16, rows=True)
    R = h.shape[0]
    if h.shape[1] != (2 * I if L.GATED[kind] else I):
        raise ValueError(f"h has {h.shape[1]} columns, {kind} of {I} needs {2 * I if L.GATED[kind] else I}")
    codes, scales = _quant_out(R, I, h.device, out)
    _call(h.device, "moe_act_fp8_quant", L.ACT[kind], h.data_ptr(), _ld(h), R, I,
          _live_ptr(slot_local_ids, R, h.device), alpha, limit, codes.data_ptr(), _ld(codes), scales.data_ptr(),
          _ld(scales))
    return codes, scales


def _w8a8_operands(A, a_scales, W, w_scales, bias, E, N, K) -> None:
    dev, G = A.device, -(-K // GROUP)
    _check(a_scales, "a_scales", _F32, (A.shape[0], G), dev, rows=True)
    lead = W.shape[:-2]
    _check(W, "W", _F8, (*lead, N, K), dev)
    _check(w_scales, "w_scales", _F32, (*lead, -(-N // GROUP), G), dev)
    if bias is not None:
        _check(bias, "bias", _BF16, (*lead, N), dev)


def moe_w8a8_gemm(A: torch.Tensor, a_scales: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                  sorted_token_ids: torch.Tensor, expert_ids: torch.Tensor, num_tokens_post_padded: torch.Tensor,
                  numel: int, top_k: int, block_m: int, bias: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, expected_slots: int = 0) -> torch.Tensor:
    """C[slot] = W[e] . A[slot // top_k] (+ bias[e]) for the live slots, with A e4m3fn [rows, K] and
    its scales [rows, ceil(K/128)] (moe_fp8_quant), W e4m3fn [E, N, K] and its scales
    [E, ceil(N/128), ceil(K/128)]; C is bf16 [numel, N].  expected_slots: slots expected to be live on
    this slice (0: all), a launch hint."""
    _check(A, "A", _F8, rows=True)
    if W.dim() != 3:
        raise ValueError(f"W must be [E, N, K], got {tuple(W.shape)}")
    E, N, K = W.shape
    if A.shape[1] != K:
        raise ValueError(f"A has {A.shape[1]} columns, W {K}")
    _w8a8_operands(A, a_scales, W, w_scales, bias, E, N, K)
    _check_align(sorted_token_ids, expert_ids, num_tokens_post_padded, numel, E, block_m, A.device)
    if out is None:
        out = torch.empty((numel, N), dtype=torch.bfloat16, device=A.device)
    else:
        _check(out, "out", _BF16, (numel, N), A.device, rows=True)
    _call(A.device, "moe_w8a8_gemm", A.data_ptr(), A.shape[0], _ld(A), a_scales.data_ptr(), _ld(a_scales), W.data_ptr(),
          w_scales.data_ptr(), None if bias is None else bias.data_ptr(), E, N, K, out.data_ptr(), _ld(out),
          sorted_token_ids.data_ptr(), expert_ids.data_ptr(), num_tokens_post_padded.data_ptr(), numel, top_k, block_m,
          expected_slots)
    return out


def moe_w8a8_linear(A: torch.Tensor, a_scales: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The same product without routing: W e4m3fn [N, K], C = A W^T (+ bias) is bf16 [M, N]."""
    _check(A, "A", _F8, rows=True)
    if W.dim() != 2:
        raise ValueError(f"W must be [N, K], got {tuple(W.shape)}")
    (M, K), N = A.shape, W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"A has {K} columns, W {W.shape[1]}")
    _w8a8_operands(A, a_scales, W, w_scales, bias, 1, N, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    else:
        _check(out, "out", _BF16, (M, N), A.device, rows=True)
    _call(A.device, "moe_w8a8_linear", A.data_ptr(), M, _ld(A), a_scales.data_ptr(), _ld(a_scales), W.data_ptr(),
          w_scales.data_ptr(), None if bias is None else bias.data_ptr(), N, K, out.data_ptr(), _ld(out))
    return out


def moe_bf16_gemm(A: torch.Tensor, W: torch.Tensor, sorted_token_ids: torch.Tensor, expert_ids: torch.Tensor,
                  num_tokens_post_padded: torch.Tensor, numel: int, top_k: int, block_m: int,
                  bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  expected_slots: int = 0, slot_local_ids: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C[slot] = W[e] . A[slot // top_k] (+ bias[e]) for the live slots: A bf16 [rows, K], W bf16
    [E, N, K], bias bf16 [E, N]; C is bf16 [numel, N].  With slot_local_ids the rows of dropped slots are
    zeroed, without they are left as they are.  expected_slots as moe_w8a8_gemm."""
    _check(A, "A", _BF16, rows=True)
    if W.dim() != 3 or W.shape[2] != A.shape[1]:
        raise ValueError(f"W {tuple(W.shape)} must be [E, N, K] with the {A.shape[1]} columns of A")
    dev, (E, N, K) = A.device, W.shape
    _check(W, "W", _BF16, dev=dev)
    if bias is not None:
        _check(bias, "bias", _BF16, (E, N), dev)
    _check_align(sorted_token_ids, expert_ids, num_tokens_post_padded, numel, E, block_m, dev)
    if out is None:
        out = torch.empty((numel, N), dtype=torch.bfloat16, device=dev)
    else:
        _check(out, "out", _BF16, (numel, N), dev, rows=True)
    _bf16_gemm(A, W, sorted_token_ids, expert_ids, num_tokens_post_padded, numel, top_k, block_m, bias, out,
               expected_slots, _live_ptr(slot_local_ids, numel, dev))
    return out


# (the calls proper, for tensors that have been checked)
def _bf16_gemm(A, W, sorted_ids, expert_ids, ntpp, numel, top_k, block_m, bias, out, expected, live) -> None:
    E, N, K = W.shape
    _call(A.device, "moe_bf16_gemm", A.data_ptr(), A.shape[0], _ld(A), W.data_ptr(),
          None if bias is None else bias.data_ptr(), E, N, K, out.data_ptr(), _ld(out), sorted_ids.data_ptr(),
          expert_ids.data_ptr(), ntpp.data_ptr(), live, numel, top_k, block_m, expected)


def _dgrad(dC, W, sorted_ids, expert_ids, ntpp, live: int, top_k, block_m, out, work, expected) -> None:
    E, N, K = W.shape
    _call(dC.device, "moe_bf16_gemm_dgrad", dC.data_ptr(), _ld(dC), W.data_ptr(), E, N, K, out.data_ptr(), _ld(out),
          sorted_ids.data_ptr(), expert_ids.data_ptr(), ntpp.data_ptr(), live, dC.shape[0], top_k, block_m, expected,
          None if work is None else work.data_ptr(), 0 if work is None else work.numel())


def _wgrad(dC, A, E, sorted_ids, expert_ids, ntpp, top_k, block_m, out, out_bias) -> None:
    dtype = (out_bias if out is None else out).dtype
    _call(dC.device, "moe_bf16_gemm_wgrad", dC.data_ptr(), _ld(dC), A.data_ptr(), A.shape[0], _ld(A), E, dC.shape[1],
          A.shape[1], None if out is None else out.data_ptr(), None if out_bias is None else out_bias.data_ptr(),
          int(dtype is torch.float32), sorted_ids.data_ptr(), expert_ids.data_ptr(), ntpp.data_ptr(), dC.shape[0], top_k,
          block_m)


def moe_bf16_gemm_dgrad(dC: torch.Tensor, W: torch.Tensor, sorted_token_ids: torch.Tensor, expert_ids: torch.Tensor,
                        num_tokens_post_padded: torch.Tensor, slot_local_ids: torch.Tensor, top_k: int, block_m: int,
                        out: Optional[torch.Tensor] = None, work: Optional[torch.Tensor] = None,
                        expected_slots: int = 0) -> torch.Tensor:
    """Gradient of moe_bf16_gemm with respect to A: dC bf16 [numel, N], W bf16 [E, N, K] -> bf16
    [numel // top_k, K], zero in rows without a live slot.  `work`: float32 workspace of numel * K
    values for top_k > 1 (allocated when not given).  expected_slots as moe_w8a8_gemm."""
    _check(dC, "dC", _BF16, rows=True)
    dev, numel = dC.device, dC.shape[0]
    if W.dim() != 3 or W.shape[1] != dC.shape[1]:
        raise ValueError(f"W {tuple(W.shape)} must be [E, N, K] with the {dC.shape[1]} columns of dC as N")
    E, N, K = W.shape
    _check(W, "W", _BF16, dev=dev)
    _check_align(sorted_token_ids, expert_ids, num_tokens_post_padded, numel, E, block_m, dev)
    if top_k < 1 or numel % top_k:
        raise ValueError(f"{numel} slots are no whole rows of top_k={top_k}")
    live = _live_ptr(slot_local_ids, numel, dev)
    if live is None:
        raise ValueError("slot_local_ids is needed: it says which slots a row's gradient sums")
    if out is None:
        out = torch.empty((numel // top_k, K), dtype=torch.bfloat16, device=dev)
    else:
        _check(out, "out", _BF16, (numel // top_k, K), dev, rows=True)
    if top_k > 1:
        if work is None:
            work = torch.empty(numel * K, dtype=torch.float32, device=dev)
        else:
            _check(work, "work", _F32, dev=dev)
    else:
        work = None
    _dgrad(dC, W, sorted_token_ids, expert_ids, num_tokens_post_padded, live, top_k, block_m, out, work,
           expected_slots)
    return out


def moe_bf16_gemm_wgrad(dC: torch.Tensor, A: torch.Tensor, n_experts: int, sorted_token_ids: torch.Tensor,
                        expert_ids: torch.Tensor, num_tokens_post_padded: torch.Tensor, top_k: int, block_m: int,
                        bias_grad: bool = False, dtype: torch.dtype = torch.bfloat16,
                        out: Optional[torch.Tensor] = None, out_bias: Optional[torch.Tensor] = None):
    """Gradients of moe_bf16_gemm with respect to W and, with bias_grad, the bias: dC bf16 [numel, N],
    A bf16 [numel // top_k, K] -> (dW [E, N, K], dbias [E, N] or None) in `dtype` (bf16 or float32),
    zero for experts without slots."""
    _check(dC, "dC", _BF16, rows=True)
    dev, (numel, N), E = dC.device, dC.shape, n_experts
    _check(A, "A", _BF16, dev=dev, rows=True)
    K = A.shape[1]
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"weight gradients are bfloat16 or float32, not {dtype}")
    _check_align(sorted_token_ids, expert_ids, num_tokens_post_padded, numel, E, block_m, dev)
    if out is None:
        out = torch.empty((E, N, K), dtype=dtype, device=dev)
    else:
        _check(out, "out", (dtype,), (E, N, K), dev)
    if bias_grad:
        if out_bias is None:
            out_bias = torch.empty((E, N), dtype=dtype, device=dev)
        else:
            _check(out_bias, "out_bias", (dtype,), (E, N), dev)
    else:
        out_bias = None
    _wgrad(dC, A, E, sorted_token_ids, expert_ids, num_tokens_post_padded, top_k, block_m, out, out_bias)
    return out, out_bias


class _ExpertsLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, A, W, bias, sorted_ids, expert_ids, ntpp, slot_local, top_k, block_m, expected):
        out = moe_bf16_gemm(A, W, sorted_ids, expert_ids, ntpp, slot_local.numel(), top_k, block_m, bias=bias,
                            expected_slots=expected, slot_local_ids=slot_local)
        ctx.save_for_backward(A, W, sorted_ids, expert_ids, ntpp, slot_local)
        ctx.top_k, ctx.block_m, ctx.expected = top_k, block_m, expected
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        A, W, *align, slot_local = ctx.saved_tensors
        # (a gradient may arrive broadcast or transposed, or with rows that 16-byte loads cannot take: between
        # 16-byte boundaries it may be contiguous already, as a part of a concatenation's is, so it is copied)
        if grad.stride(-1) != 1 or grad.stride(0) % 8 or grad.stride(0) < grad.shape[1] or grad.data_ptr() % 16:
            grad = grad.clone(memory_format=torch.contiguous_format)
        dA = dW = db = None
        if ctx.needs_input_grad[0]:
            dA = torch.empty(A.shape, dtype=A.dtype, device=A.device)
            work = None if ctx.top_k == 1 else torch.empty(grad.shape[0] * W.shape[2], dtype=torch.float32, device=A.device)
            _dgrad(grad, W, *align, slot_local.data_ptr(), ctx.top_k, ctx.block_m, dA, work, ctx.expected)
        if ctx.needs_input_grad[1] or ctx.needs_input_grad[2]:
            if ctx.needs_input_grad[1]:
                dW = torch.empty_like(W)
            if ctx.needs_input_grad[2]:
                db = torch.empty(W.shape[:2], dtype=W.dtype, device=W.device)
            _wgrad(grad, A, W.shape[0], *align, ctx.top_k, ctx.block_m, dW, db)
        return dA, dW, db, None, None, None, None, None, None, None


def moe_experts_linear(A: torch.Tensor, W: torch.Tensor, align, top_k: int, block_m: int,
                       bias: Optional[torch.Tensor] = None, expected_slots: int = 0) -> torch.Tensor:
    """Differentiable moe_bf16_gemm: C bf16 [numel, N] with C[slot] = W[e] . A[slot // top_k]
    (+ bias[e]) and zeros in the rows of dropped slots.

    `align` is what moe_align returns for the batch (sorted_token_ids, expert_ids,
    num_tokens_post_padded, slot_local_ids) with the same block_m; A has numel // top_k rows (one
    for each token with the layer's top_k, or one for each slot with top_k = 1).  Gradients flow to
    A, W and bias; they are bf16, once differentiable, and zero for rows and experts without slots.
    expected_slots as moe_w8a8_gemm.

    The align's tensors are kept for the backward pass: buffers that a later batch's align writes over
    must not be among them.  The forward and the backward pass can be captured into a graph.  As with
    any autograd work, hold no graph of an eager call of the same leaves while capturing: torch then
    waits on the eager call's stream inside the capture, which ends the process."""
    sorted_ids, expert_ids, ntpp, slot_local = align
    if slot_local is None:
        raise ValueError("moe_experts_linear needs the align's slot_local_ids")
    if top_k < 1 or A.dim() != 2 or A.shape[0] * top_k != slot_local.numel():
        raise ValueError(f"A {tuple(A.shape)} must have a row for each {top_k} of the {slot_local.numel()} slots")
    return _ExpertsLinear.apply(A, W, bias, sorted_ids, expert_ids, ntpp, slot_local, top_k, block_m, expected_slots)
