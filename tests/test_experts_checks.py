"""Refusals of the products with 8-bit and bf16 expert weights and of the quantiser: the C entry
points validate on the host before anything is launched, so they are called here with addresses
that are never used."""
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from quantized_mixture_experts_align_amd import _lib as L

A16 = 0x10000          # an aligned address
QUANT = dict(x=A16, ld_x=256, R=4, K=256, live=None, codes=A16, ld_codes=256, scales=A16, ld_scales=2, stream=None)
W8A8 = dict(A=A16, a_rows=8, lda=256, a_scales=A16, ld_scales=2, W=A16, w_scales=A16, bias=None, E=4, N=128, K=256,
            C=A16, ldc=128, sorted=A16, eids=A16, ntpp=A16, numel=16, top_k=2, block_m=16, expected=0, stream=None)
LINEAR = dict(A=A16, M=8, lda=256, a_scales=A16, ld_scales=2, W=A16, w_scales=A16, bias=None, N=128, K=256, C=A16,
              ldc=128, stream=None)
BF16 = dict(A=A16, a_rows=8, lda=256, W=A16, bias=None, E=4, N=128, K=256, C=A16, ldc=128, sorted=A16, eids=A16,
            ntpp=A16, live=None, numel=16, top_k=2, block_m=16, expected=0, stream=None)
DGRAD = dict(dC=A16, ld_dc=128, W=A16, E=4, N=128, K=256, dA=A16, ld_da=256, sorted=A16, eids=A16, ntpp=A16, live=A16,
             numel=16, top_k=2, block_m=16, expected=0, work=A16, work_elems=16 * 256, stream=None)
WGRAD = dict(dC=A16, ld_dc=128, A=A16, a_rows=8, lda=256, E=4, N=128, K=256, dW=A16, dbias=None, f32=0, sorted=A16,
             eids=A16, ntpp=A16, numel=16, top_k=2, block_m=16, stream=None)

BAD = [
    ("moe_fp8_quant", QUANT, L.MOE_EINVAL, [dict(x=None), dict(codes=None), dict(scales=None), dict(R=-1), dict(K=0),
                                            dict(ld_x=128), dict(ld_codes=248), dict(ld_scales=1)]),
    ("moe_fp8_quant", QUANT, L.MOE_EUNSUPPORTED, [dict(K=252), dict(ld_x=260), dict(ld_codes=260), dict(x=A16 + 8),
                                                  dict(codes=A16 + 4), dict(scales=A16 + 2), dict(R=1 << 30)]),
    ("moe_w8a8_gemm", W8A8, L.MOE_EINVAL, [dict(A=None), dict(W=None), dict(C=None), dict(a_scales=None),
                                           dict(w_scales=None), dict(sorted=None), dict(eids=None), dict(ntpp=None),
                                           dict(E=0), dict(N=0), dict(K=0), dict(numel=-1), dict(top_k=0),
                                           dict(block_m=0), dict(block_m=257), dict(a_rows=7), dict(lda=240),
                                           dict(lda=264), dict(ldc=120), dict(ldc=130), dict(ld_scales=1)]),
    ("moe_w8a8_gemm", W8A8, L.MOE_EUNSUPPORTED, [dict(E=513), dict(N=124), dict(K=248), dict(A=A16 + 8),
                                                 dict(W=A16 + 8), dict(C=A16 + 4), dict(bias=A16 + 4),
                                                 dict(a_scales=A16 + 2), dict(numel=1 << 30, a_rows=1 << 30)]),
    ("moe_w8a8_linear", LINEAR, L.MOE_EINVAL, [dict(A=None), dict(W=None), dict(C=None), dict(a_scales=None),
                                               dict(w_scales=None), dict(M=-1), dict(lda=128), dict(ldc=64),
                                               dict(ld_scales=1)]),
    ("moe_w8a8_linear", LINEAR, L.MOE_EUNSUPPORTED, [dict(N=132), dict(K=264, lda=272), dict(A=A16 + 4)]),
    ("moe_bf16_gemm", BF16, L.MOE_EINVAL, [dict(A=None), dict(W=None), dict(C=None), dict(sorted=None), dict(eids=None),
                                           dict(ntpp=None), dict(E=0), dict(a_rows=7), dict(lda=248), dict(lda=260),
                                           dict(ldc=124), dict(top_k=0), dict(block_m=300)]),
    ("moe_bf16_gemm", BF16, L.MOE_EUNSUPPORTED, [dict(E=600), dict(N=130, ldc=132), dict(K=252), dict(A=A16 + 2),
                                                 dict(W=A16 + 2), dict(C=A16 + 2), dict(bias=A16 + 2)]),
    ("moe_bf16_gemm_dgrad", DGRAD, L.MOE_EINVAL, [dict(dC=None), dict(W=None), dict(dA=None), dict(sorted=None),
                                                  dict(eids=None), dict(ntpp=None), dict(live=None), dict(work=None),
                                                  dict(ld_dc=120), dict(ld_dc=132), dict(ld_da=248), dict(ld_da=260),
                                                  dict(numel=15), dict(E=0), dict(block_m=0)]),
    ("moe_bf16_gemm_dgrad", DGRAD, L.MOE_EUNSUPPORTED, [dict(dC=A16 + 8), dict(W=A16 + 8), dict(dA=A16 + 8),
                                                        dict(work=A16 + 8), dict(N=132, ld_dc=136), dict(E=513)]),
    ("moe_bf16_gemm_dgrad", DGRAD, L.MOE_ESIZE, [dict(work_elems=16 * 256 - 1)]),
    ("moe_bf16_gemm_wgrad", WGRAD, L.MOE_EINVAL, [dict(dC=None), dict(A=None), dict(dW=None), dict(sorted=None),
                                                  dict(eids=None), dict(ntpp=None), dict(a_rows=7), dict(lda=248),
                                                  dict(numel=17), dict(ld_dc=64), dict(top_k=0)]),
    ("moe_bf16_gemm_wgrad", WGRAD, L.MOE_EUNSUPPORTED, [dict(A=A16 + 8), dict(dW=A16 + 8), dict(dbias=A16 + 2),
                                                        dict(K=260, lda=264), dict(E=513)]),
]


@pytest.mark.parametrize("name,good,code,changes", BAD, ids=[f"{b[0]}-{-b[2]}" for b in BAD])
def test_entry_points_refuse(name, good, code, changes):
    f = getattr(L.lib(), name)
    for change in changes:
        args = {**good, **change}
        assert list(args) == list(good)
        assert f(*args.values()) == code, change
        assert name.encode() in L.lib().moe_last_error(), change


def test_activation_kinds_are_checked():
    f = L.lib().moe_act_fp8_quant
    assert f(7, A16, 512, 4, 256, None, 1.0, 1.0, A16, 256, A16, 2, None) == L.MOE_EINVAL
    assert f(0, A16, 504, 4, 256, None, 1.0, 1.0, A16, 256, A16, 2, None) == L.MOE_EINVAL     # 2I columns for a gate
    with pytest.raises(ValueError, match="unknown activation"):
        P.moe_act_fp8_quant("gelu", torch.zeros((2, 16), dtype=torch.bfloat16), 8)


def test_empty_batches_launch_nothing():
    for name, good, change in (("moe_fp8_quant", QUANT, dict(R=0, x=None, codes=None)),
                               ("moe_w8a8_gemm", W8A8, dict(numel=0, A=None, C=None, sorted=None)),
                               ("moe_w8a8_linear", LINEAR, dict(M=0, A=None)),
                               ("moe_bf16_gemm", BF16, dict(numel=0, A=None)),
                               ("moe_bf16_gemm_dgrad", DGRAD, dict(numel=0, dC=None, dA=None, work_elems=0))):
        assert getattr(L.lib(), name)(*{**good, **change}.values()) == L.MOE_OK, name


def test_host_tensors_are_refused():
    x, i = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros(16, dtype=torch.int32)
    q, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1))
    w = torch.zeros((1, 128, 128), dtype=torch.bfloat16)
    for call in (lambda: P.moe_fp8_quant(x), lambda: P.moe_act_fp8_quant("relu2", x, 128),
                 lambda: P.moe_w8a8_linear(q, s, q, s), lambda: P.moe_w8a8_gemm(q, s, w, s, i, i, i, 4, 1, 16),
                 lambda: P.moe_bf16_gemm(x, w, i, i, i, 4, 1, 16), lambda: P.moe_bf16_gemm_dgrad(x, w, i, i, i, i, 1, 16),
                 lambda: P.moe_bf16_gemm_wgrad(x, x, 1, i, i, i, 1, 16)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_experts_linear_checks_its_rows():
    align = (None, None, None, torch.zeros((4, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="must have a row"):
        P.moe_experts_linear(torch.zeros((3, 8)), torch.zeros((1, 8, 8)), align, 2, 16)
    with pytest.raises(ValueError, match="slot_local_ids"):
        P.moe_experts_linear(torch.zeros((4, 8)), torch.zeros((1, 8, 8)), (None, None, None, None), 2, 16)


def test_the_bias_gradient_alone_needs_no_rows():
    f = L.lib().moe_bf16_gemm_wgrad
    alone = {**WGRAD, **dict(A=None, a_rows=0, lda=0, dW=None, dbias=A16)}
    for change, code in ((dict(dbias=A16 + 2), L.MOE_EUNSUPPORTED), (dict(dbias=None), L.MOE_EINVAL),
                         (dict(ntpp=None), L.MOE_EINVAL), (dict(dC=None), L.MOE_EINVAL), (dict(ld_dc=120), L.MOE_EINVAL)):
        assert f(*{**alone, **change}.values()) == code, change


# A launch has fewer than 2^32 threads: streamed blocks; tiles of 32 to 256 rows; the sum over a row's slots
@pytest.mark.parametrize("name,good,change", [
    ("moe_bf16_gemm", BF16, dict(numel=1 << 25, a_rows=1 << 25, N=8192, ldc=8192)),
    ("moe_w8a8_gemm", W8A8, dict(numel=1 << 25, a_rows=1 << 25, N=8192, ldc=8192)),
    ("moe_bf16_gemm", BF16, dict(numel=1 << 28, a_rows=1 << 28, N=8192, ldc=8192, block_m=32)),
    ("moe_bf16_gemm", BF16, dict(numel=1 << 29, a_rows=1 << 29, N=8192, ldc=8192, block_m=128)),
    ("moe_w8a8_linear", LINEAR, dict(M=1 << 29, N=8192, ldc=8192)),
    ("moe_bf16_gemm_dgrad", DGRAD, dict(numel=1 << 26, N=8, K=8, ld_dc=8, ld_da=8, block_m=256, work_elems=1 << 29)),
    ("moe_bf16_gemm_dgrad", DGRAD, dict(numel=1 << 29, N=8, K=8192, ld_dc=8, ld_da=8192, top_k=1, block_m=64))])
def test_launches_of_too_many_threads_are_refused(name, good, change):
    assert getattr(L.lib(), name)(*{**good, **change}.values()) == L.MOE_EUNSUPPORTED
    assert b"grid too large" in L.lib().moe_last_error()
