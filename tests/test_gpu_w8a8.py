"""moe_w8a8_gemm and moe_w8a8_linear against the 64-bit product of the dequantised operands."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests.experts_util import U16, U32, aligned, assert_close, bf16, e4m3, product8, routing, scales, spread, strided

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


def cancelling(rows, E, N, K, seed):
    """Operands of small whole numbers whose groups cancel in pairs up to their scales: A holds a group and its
    negative, W the same group twice, and the scales of a pair differ by at most 2^-10 of themselves."""
    r = np.random.default_rng([seed, 81])
    G = K // 128
    whole = lambda *s: r.integers(-2, 3, s).astype(np.float32)                    # noqa: E731
    near = lambda s: np.stack([s, s * (1 + r.uniform(-1, 1, s.shape) / 1024)], -1).astype(np.float32)  # noqa: E731
    a, w = whole(rows, G // 2, 128), whole(E, N, G // 2, 128)
    A = np.stack([a, -a], 2).reshape(rows, K)
    W = np.stack([w, w], 3).reshape(E, N, K)
    sa = near(np.exp(r.normal(-5, 1, (rows, G // 2)))).reshape(rows, G)
    sb = near(np.exp(r.normal(-5, 1, (E, -(-N // 128), G // 2)))).reshape(E, -1, G)
    f8 = lambda t: torch.from_numpy(t).to(torch.float8_e4m3fn)                    # noqa: E731
    return f8(A), torch.from_numpy(sa), f8(W), torch.from_numpy(sb)


def assert_scaled_in_fp32(got, a, sa, w, sb, local, top_k):
    """Sums of whole products are exact in every order (at most 4 * 128 for a group, and eight products of which
    the largest is 4 and the least 1 lose nothing in the matrix instruction).  What is left is the rounding of
    sa * sb and one for each group added, and at most eight for joining parts of K: each at most u32 of the sum
    of the groups' magnitudes S.  The result is some 2^-10 of S, so that a relative error of 2^-17 in a group
    stands out from the result's own rounding to bf16."""
    G = a.shape[1] // 128
    N = w.shape[1]
    for e in range(w.shape[0]):
        s = np.flatnonzero(local == e)
        C, S = np.zeros((len(s), N)), np.zeros((len(s), N))
        A, B = a[s // top_k].double().numpy(), w[e].double().numpy()
        row, block = sa[s // top_k].double().numpy(), np.repeat(sb[e].double().numpy(), 128, 0)[:N]
        for g in range(G):
            part = np.outer(row[:, g], block[:, g]) * (A[:, g * 128: (g + 1) * 128] @ B[:, g * 128: (g + 1) * 128].T)
            C += part
            S += np.abs(part)
        assert_close(got[torch.from_numpy(s).to(got.device)], C,
                     (G + 9) * U32 * S * (1 + U16) + U16 * np.abs(C) + 1e-30, f"C of expert {e}")


@pytest.mark.parametrize("M,k,E,N,K,B", [
    (4, 2, 4, 264, 4096, 16), (8, 2, 8, 1032, 512, 16), (200, 2, 8, 520, 512, 16), (450, 2, 64, 520, 512, 16),
    (100, 2, 4, 4104, 4096, 7), (400, 2, 8, 4096, 512, 32), (40, 2, 2, 264, 1024, 32), (400, 2, 8, 4096, 512, 64),
    (60, 2, 2, 264, 1024, 64), (1792, 2, 4, 2048, 512, 128), (1792, 2, 4, 2048, 2048, 128), (200, 2, 2, 520, 512, 128),
    (1500, 2, 3, 4104, 512, 256), (5500, 2, 3, 1032, 512, 128)])
def test_block_scales_are_applied_in_fp32(M, k, E, N, K, B):
    al, local = aligned(routing(M, k, E + 1, E, M), 0, E, B)
    a, sa, w, sb = cancelling(M, E, N, K, M + B)
    got = P.moe_w8a8_gemm(a.cuda(), sa.cuda(), w.cuda(), sb.cuda(), *al[:3], M * k, k, B)
    assert_scaled_in_fp32(got, a, sa, w, sb, local, k)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (3, 136, 512), (20, 520, 1024), (64, 264, 2048), (300, 1032, 512),
                                   (3000, 4104, 512)])
def test_block_scales_of_the_dense_product(M, N, K):
    a, sa, w, sb = cancelling(M, 1, N, K, M + N)
    got = P.moe_w8a8_linear(a.cuda(), sa.cuda(), w[0].cuda(), sb[0].cuda())
    assert_scaled_in_fp32(got, a, sa, w, sb, np.zeros(M, np.int64), 1)


def without_quantisation(x, w13, s13, w2, s2, gw, local):
    """The layer (silu) of unquantised activations in 64 bits [M, H], and the size (2-norm over all of it) of
    what quantising them to e4m3 does to it, to first order.

    A rounding to e4m3 is off by at most 2^-4 of the value, 2^-4 / sqrt(3) in the root mean square, and independent
    of the others: a sum of products p is then off by 2^-4 / sqrt(3) * sqrt(sum p^2).  For an activation
    silu(g) * u that is slope(g) |u| times g's, |silu(g)| times u's, and its own rounding; the three are added as
    if they always had the same sign, which covers the bf16 roundings between the stages (2^-9 each) too."""
    H, I, k = w2.shape[1], w2.shape[2], gw.shape[1]
    a13, a2 = w13.double().numpy() * spread(s13, 2 * I, H), w2.double().numpy() * spread(s2, H, I)
    x64, c = x.double().numpy(), gw.double().numpy().reshape(-1)
    plain, square = np.zeros((len(x64), H)), 0.0
    for s in np.flatnonzero(local >= 0):
        w, v = a13[local[s]], x64[s // k]
        h, dh = w @ v, np.sqrt(w ** 2 @ v ** 2)
        g, u, t = h[:I], h[I:], 1 / (1 + np.exp(-h[:I]))
        plain[s // k] += c[s] * (a2[local[s]] @ (g * t * u))
        d = np.abs(t * (1 + g * (1 - t)) * u) * dh[:I] + np.abs(g * t) * dh[I:] + np.abs(g * t * u)
        square += (c[s] ** 2 * (a2[local[s]] ** 2 @ d ** 2)).sum()
    return plain, 2.0 ** -4 / np.sqrt(3) * np.sqrt(square)


@pytest.mark.parametrize("B", [16, 32, 128])
def test_each_stage_of_the_layer_of_8_bit_experts(B):
    """quantise -> gate/up -> activation and quantise -> down -> combine on a slice of the experts: each stage
    against 64 bits of what the stage in front gave it, and the end against the layer without quantisation."""
    M, k, E, H, I = 96, 2, 4, 384, 256
    ids = routing(M, k, E + 1, E, 31)                                  # expert E is elsewhere
    al, local = aligned(ids, 0, E, B)
    x = bf16((M, H), 32)
    w13, s13 = e4m3((E, 2 * I, H), 33), scales((E, 2 * I // 128, H // 128), 33) * 0.02
    w2, s2 = e4m3((E, H, I), 34), scales((E, H // 128, I // 128), 34) * 0.02
    gw = torch.from_numpy(np.random.default_rng(35).random((M, k), dtype=np.float32))
    on = np.flatnonzero(local >= 0)
    half_step = lambda v, s: np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s) * (1 + 2.0 ** -18)   # noqa: E731

    q, qs = P.moe_fp8_quant(x.cuda())
    back = lambda c, s, n: c.double().cpu().numpy() * spread(s.cpu(), c.shape[0], n)                # noqa: E731
    x64 = x.double().numpy()
    assert (np.abs(back(q, qs, H) - x64) <= half_step(x64, np.repeat(qs.double().cpu().numpy(), 128, 1))).all()

    h = P.moe_w8a8_gemm(q, qs, w13.cuda(), s13.cuda(), *al[:3], M * k, k, B)
    want, bound = product8(q.cpu(), qs.cpu(), w13, s13, None, local, k)
    assert_close(h[torch.from_numpy(on).cuda()], want[on], (bound + U16 * np.abs(want) + 1e-30)[on], "gate/up")

    c, cs = P.moe_act_fp8_quant("silu_mul", h, I, al[3])
    h64 = h.double().cpu().numpy()[on]
    act = h64[:, :I] / (1 + np.exp(-h64[:, :I])) * h64[:, I:]
    # (the activation in fp32: under 2^-18 relative)
    off = np.abs(back(c, cs, I)[on] - act)
    assert (off <= half_step(act, np.repeat(cs.double().cpu().numpy()[on], 128, 1)) + 2.0 ** -17 * np.abs(act)).all()

    y = P.moe_w8a8_gemm(c, cs, w2.cuda(), s2.cuda(), *al[:3], M * k, 1, B)
    c0, cs0 = c.cpu(), cs.cpu()
    c0.view(torch.uint8)[local < 0], cs0[local < 0] = 0, 0             # (what dropped rows hold is not written)
    want, bound = product8(c0, cs0, w2, s2, None, local, 1)
    assert_close(y[torch.from_numpy(on).cuda()], want[on], (bound + U16 * np.abs(want) + 1e-30)[on], "down")

    out = P.moe_combine(y, gw.cuda(), al[3])
    y64 = np.where((local >= 0)[:, None], np.nan_to_num(y.double().cpu().numpy()), 0.0).reshape(M, k, H)
    terms = gw.double().numpy()[..., None] * y64
    want = terms.sum(1)
    assert_close(out, want, (k + 1) * U32 * np.abs(terms).sum(1) * (1 + U16) + U16 * np.abs(want) + 1e-30, "combine")

    plain, err = without_quantisation(x, w13, s13, w2, s2, gw, local)
    off = np.linalg.norm(out.double().cpu().numpy() - plain)
    assert off <= err, (off, err)
