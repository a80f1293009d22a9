"""moe_w8a8_gemm and moe_w8a8_linear against the 64-bit product of the dequantised operands."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests.experts_util import U16, aligned, assert_close, bf16, e4m3, product8, routing, scales, spread, strided

pytestmark = pytest.mark.gpu

NANS = 0x7F


def case(M, k, E_all, E, N, K, B, top_k, bias, seed, start=0, only=None, pad=0, expected=0):
    ids = routing(M, k, E_all, E, seed, only)
    al, local = aligned(ids, start, E, B)
    rows = M if top_k == k else M * k
    a, sa = e4m3((rows, K), seed), scales((rows, -(-K // 128)), seed)
    w, sb = e4m3((E, N, K), seed + 1), scales((E, -(-N // 128), -(-K // 128)), seed + 1)
    b = bf16((E, N), seed + 2) if bias else None
    want, bound = product8(a, sa, w, sb, None if b is None else b.double().numpy(), local, top_k)
    A = strided(a.view(torch.uint8).float(), K + pad, NANS).to(torch.uint8) if pad else a.cuda()
    SA = strided(sa, sa.shape[1] + 3) if pad else sa.cuda()
    base = torch.full((M * k, N + (8 if pad else 0)), -5.0, dtype=torch.bfloat16, device="cuda")
    out = base[:, :N]
    got = P.moe_w8a8_gemm(A, SA, w.cuda(), sb.cuda(), *al[:3], M * k, top_k, B, bias=None if b is None else b.cuda(),
                          out=out, expected_slots=expected)
    assert got is out
    dead = local < 0
    assert bool((base[torch.from_numpy(dead).cuda()] == -5.0).all()) and bool((base[:, N:] == -5.0).all())
    live = np.flatnonzero(~dead)
    assert_close(got[torch.from_numpy(live).cuda()], want[live], bound[live] + U16 * np.abs(want[live]) + 1e-30, "C")
    return got


@pytest.mark.parametrize("B", [1, 7, 16, 32, 64, 100, 128, 256])
def test_block_sizes(B):
    case(53, 2, 6, 6, 264, 400, B, 2, True, 100 + B)


@pytest.mark.parametrize("M,k,E,N,K,B", [
    (1, 1, 1, 8, 16, 16), (1, 2, 8, 2048, 512, 16), (3, 4, 16, 2880, 2880, 16), (7, 2, 4, 136, 128, 32),
    (300, 2, 4, 512, 1024, 64), (513, 4, 8, 1032, 272, 128), (640, 2, 5, 768, 144, 128), (130, 1, 2, 24, 4112, 64),
    (1025, 1, 1, 520, 256, 128), (200, 3, 12, 264, 1152, 32)])
@pytest.mark.parametrize("gather", [True, False])
def test_shapes(M, k, E, N, K, B, gather):
    case(M, k, E, E, N, K, B, k if gather else 1, M % 2 == 1, M + N + K)


@pytest.mark.parametrize("M,k,E,N,K,B", [(1100, 1, 2, 520, 400, 128), (2100, 2, 8, 264, 272, 128), (700, 2, 2, 1032, 256, 256),
                                         (5000, 1, 3, 2056, 144, 128), (4200, 1, 1, 4104, 128, 128)])
def test_tiles_of_several_blocks(M, k, E, N, K, B):
    # enough slots an expert for 256-row tiles, made of two 128-row blocks or of one of 256; skewed, so
    # that experts end inside a tile, in its first block, or have no slot
    r = np.random.default_rng(M)
    case(M, k, 2 * E, E, N, K, B, k, True, M, only=r.choice(2 * E, size=max(k, E), replace=False))
    case(M, k, E, E, N, K, B, 1, False, M + 1, only=[E - 1] if k == 1 else None)


@pytest.mark.parametrize("B", [16, 32, 128])
@pytest.mark.parametrize("expected", [1, 40, 100000])
def test_the_launch_hint_changes_no_result(B, expected):
    case(130, 4, 5, 5, 520, 656, B, 4, False, 70 + B, expected=expected)


@pytest.mark.parametrize("B", [16, 64, 128])
def test_slice_strides_and_what_lies_behind_rows(B):
    # a slice of the experts (most slots dropped), rows of A and of the output apart with NaN codes
    # and NaN scales between them
    case(150, 4, 24, 6, 200, 336, B, 4, True, 9, start=5, pad=48)


@pytest.mark.parametrize("B", [16, 128])
def test_empty_experts_and_nothing_local(B):
    case(40, 2, 9, 9, 128, 256, B, 2, False, 21, only=[2, 7])          # all tokens on two experts
    case(40, 2, 9, 3, 128, 256, B, 2, False, 22, only=[5, 6, 8])       # none in the slice
    case(200, 1, 4, 4, 128, 256, B, 1, False, 23, only=[3])            # all on the last one


def test_no_tokens():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    al = P.moe_align(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 0, 4, 16)
    out = P.moe_w8a8_gemm(e4m3((0, 128), 1).cuda(), scales((0, 1), 1).cuda(), e4m3((4, 64, 128), 1).cuda(),
                          scales((4, 1, 1), 1).cuda(), *al[:3], 0, 2, 16)
    assert out.shape == (0, 64) and z.numel() == 0
    assert P.moe_w8a8_linear(e4m3((0, 128), 1).cuda(), scales((0, 1), 1).cuda(), e4m3((64, 128), 1).cuda(),
                             scales((1, 1), 1).cuda()).shape == (0, 64)


@pytest.mark.parametrize("B", [16, 128])
def test_a_nan_code_stays_in_its_row_and_column(B):
    M, N, K, E = 140, 136, 272, 2
    ids = routing(M, 1, E, E, 4)
    al, local = aligned(ids, 0, E, B)
    a, w = e4m3((M, K), 5).view(torch.uint8), e4m3((E, N, K), 6).view(torch.uint8)
    a[17, 271] = NANS
    w[1, 40, 0] = NANS
    out = P.moe_w8a8_gemm(a.cuda(), scales((M, 3), 5).cuda(), w.cuda(), scales((E, 2, 3), 6).cuda(), *al[:3], M, 1, B)
    nan = torch.isnan(out.float()).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[17] = True
    want[local == 1, 40] = True
    assert np.array_equal(nan, want)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 7168), (2, 8, 16), (17, 1000, 528), (64, 264, 2880), (129, 1032, 384),
                                   (777, 640, 1040), (2049, 264, 256)])
@pytest.mark.parametrize("bias", [False, True])
def test_linear(M, N, K, bias):
    a, sa = e4m3((M, K), M), scales((M, -(-K // 128)), M)
    w, sb = e4m3((1, N, K), N), scales((1, -(-N // 128), -(-K // 128)), N)
    b = bf16((1, N), K) if bias else None
    want, bound = product8(a, sa, w, sb, None if b is None else b.double().numpy(), np.zeros(M, np.int64), 1)
    got = P.moe_w8a8_linear(strided(a.view(torch.uint8).float(), K + 16, NANS).to(torch.uint8), sa.cuda(), w[0].cuda(),
                            sb[0].cuda(), bias=None if b is None else b[0].cuda())
    assert_close(got, want, bound + U16 * np.abs(want) + 1e-30, "C")


def test_the_layer_of_8_bit_experts_runs_and_replays():
    """quantise -> gate/up -> activation and quantise -> down -> combine, against 64 bits with the
    same intermediate roundings left out, eagerly and as a captured graph on another stream."""
    M, k, E, H, I, B = 96, 2, 4, 384, 256, 32
    ids = routing(M, k, E, E, 31)
    x = bf16((M, H), 32)
    w13, s13 = e4m3((E, 2 * I, H), 33), scales((E, 2 * I // 128, H // 128), 33) * 0.02
    w2, s2 = e4m3((E, H, I), 34), scales((E, H // 128, I // 128), 34) * 0.02
    gw = torch.from_numpy(np.random.default_rng(35).random((M, k), dtype=np.float32))
    X, IDS, GW = x.cuda(), torch.from_numpy(ids).cuda(), gw.cuda()
    W13, S13, W2, S2 = w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda()

    def layer():
        s, e, n, loc = P.moe_align(IDS, 0, E, B)
        q, qs = P.moe_fp8_quant(X)
        h = P.moe_w8a8_gemm(q, qs, W13, S13, s, e, n, M * k, k, B)
        c, cs = P.moe_act_fp8_quant("silu_mul", h, I, loc)
        y = P.moe_w8a8_gemm(c, cs, W2, S2, s, e, n, M * k, 1, B)
        return P.moe_combine(y, GW, loc)

    first = layer().clone()
    x64, want = x.double().numpy(), np.zeros((M, H))
    size = np.zeros((M, H))
    a13, a2 = w13.double().numpy() * spread(s13, 2 * I, H), w2.double().numpy() * spread(s2, H, I)
    for t in range(M):
        for j in range(k):
            h = a13[ids[t, j]] @ x64[t]
            act = h[:I] / (1 + np.exp(-h[:I])) * h[I:]
            want[t] += gw[t, j].item() * (a2[ids[t, j]] @ act)
            size[t] += gw[t, j].item() * np.linalg.norm(a2[ids[t, j]], axis=1) * np.linalg.norm(act)
    # two quantisations to e4m3 of independent sign: each term is off by at most 2^-4, a sum of them
    # by about 2^-4 / sqrt(3) of the norm product; six of these and the bf16 roundings inside
    assert (np.abs(first.double().cpu().numpy() - want) <= 6 * 2.0 ** -4 / np.sqrt(3) * size).all()

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = layer()
    for seed in (41, 42, 43):
        X.copy_(bf16((M, H), seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, layer())
