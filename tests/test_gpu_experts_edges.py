"""The products over experts and their gradients where a launch changes its kernel or its indexes
grow: every tile shape, many blocks and many tiles a workgroup, rows that are not 16-byte aligned,
operands of more than 4 GB, align outputs with stale entries behind the live ones, calls on two
streams, and captured calls whose routing changes between replays."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests.experts_util import (ADD, U16, U32, aligned, assert_close, bf16, e4m3, product, product8, routing, scales,
                                strided)

pytestmark = pytest.mark.gpu


def skewed(M, k, E, seed):
    """Routing whose experts get from no slot at all (expert 1) to half of them."""
    r = np.random.default_rng([seed, 5])
    p = 0.5 ** np.arange(1, E + 1)
    if E > 2:
        p[1] = 0
    return r.choice(E, size=(M, k), p=p / p.sum()).astype(np.int32)


# (M, k, E, N, K of bf16 values, B): sizes for which the launch takes, in turn, streamed blocks one by one with
# K over eight waves (few of them; long rows of bf16) and over four, in pairs (odd and even counts of them, short
# blocks), 16-row blocks in 32-row tiles, 64 x 256 tiles of blocks of 32 and of 64, 128 x 128, 128 x 256,
# 256 x 256 of one block and of several (more blocks than a wave looks through at once), and tiles of an
# expert's last block
TILES = [(4, 2, 4, 264, 1544, 16), (8, 2, 8, 1032, 3112, 16), (16, 2, 16, 1032, 136, 16), (200, 2, 8, 520, 72, 16),
         (120, 4, 8, 392, 136, 5), (450, 2, 64, 520, 136, 16), (400, 2, 8, 4096, 264, 32), (400, 2, 8, 4096, 264, 64),
         (1792, 2, 4, 2048, 256, 128), (1792, 2, 4, 2048, 1024, 128), (1500, 2, 3, 4104, 136, 256),
         (5500, 2, 3, 1032, 136, 128), (15000, 1, 3, 264, 72, 128)]


@pytest.mark.parametrize("M,k,E,N,K,B", TILES)
@pytest.mark.parametrize("top", [1, 0])
def test_bf16_product_and_rows_gradient(M, k, E, N, K, B, top):
    """top: A has a row for each slot (1) or for each token (0); the output's rows are 8-byte aligned; slots of
    expert E are dropped."""
    top_k = top or k
    al, local = aligned(skewed(M, k, E + 1, M), 0, E, B)
    a, w, b = bf16((M * k // top_k, K), M), bf16((E, N, K), N), bf16((E, N), K)
    W, base = w.cuda(), torch.full((M * k, N + 4), -5.0, dtype=torch.bfloat16, device="cuda")
    P.moe_bf16_gemm(a.cuda(), W, *al[:3], M * k, top_k, B, bias=b.cuda(), out=base[:, :N], slot_local_ids=al[3])
    A64, W64 = a.double().numpy(), w.double().numpy()
    want, bound = product(A64, W64, b.double().numpy(), local, top_k)
    assert_close(base[:, :N], want, bound + U16 * np.abs(want) + 1e-30, "C")
    assert bool((base[:, N:] == -5.0).all())
    # the gradient of A is the same product with W transposed, summed over a row's slots
    g = bf16((M * k, K), M + 1)
    Wt = w.transpose(1, 2).contiguous().cuda()                       # [E, K, N]: N columns of the gradient
    per_slot, bound = product(g.double().numpy(), W64, None, local, 1)
    rows = per_slot.reshape(-1, top_k, N).sum(1)
    limit = bound.reshape(-1, top_k, N).sum(1) + top_k * ADD * np.abs(per_slot).reshape(-1, top_k, N).sum(1)
    got = P.moe_bf16_gemm_dgrad(g.cuda(), Wt, *al, top_k, B)
    assert_close(got, rows, limit * (1 + U16) + U16 * np.abs(rows) + 1e-30, "dA")


@pytest.mark.parametrize("M,k,E,N,K,B", TILES)
def test_w8a8_product(M, k, E, N, K, B):
    K *= 2                                                           # the same bytes
    al, local = aligned(skewed(M, k, E, M), 0, E, B)
    G = -(-K // 128)
    a, sa, w, sb = e4m3((M, K), M), scales((M, G), M), e4m3((E, N, K), N), scales((E, -(-N // 128), G), N)
    base = torch.full((M * k, N + 4), -5.0, dtype=torch.bfloat16, device="cuda")
    P.moe_w8a8_gemm(a.cuda(), sa.cuda(), w.cuda(), sb.cuda(), *al[:3], M * k, k, B, out=base[:, :N])
    want, bound = product8(a, sa, w, sb, None, local, k)
    assert_close(base[:, :N], want, bound + U16 * np.abs(want) + 1e-30, "C")
    assert bool((base[:, N:] == -5.0).all())


def test_linear_of_256_row_tiles():
    M, N, K = 3000, 4104, 272
    a, sa, w, sb = e4m3((M, K), 1), scales((M, 3), 1), e4m3((1, N, K), 2), scales((1, 33, 3), 2)
    got = P.moe_w8a8_linear(a.cuda(), sa.cuda(), w[0].cuda(), sb[0].cuda())
    want, bound = product8(a, sa, w, sb, None, np.zeros(M, np.int32), 1)
    assert_close(got, want, bound + U16 * np.abs(want) + 1e-30, "C")


# 256 x 256 tiles and 128 x 128 ones, of which a workgroup computes several; experts of no, one and many steps
@pytest.mark.parametrize("M,k,E,N,K,B,top_k", [(900, 2, 100, 264, 520, 16, 2), (700, 3, 60, 264, 264, 32, 3),
                                               (900, 2, 100, 520, 264, 64, 1)])
def test_weight_gradients_of_many_tiles(M, k, E, N, K, B, top_k):
    r = np.random.default_rng(M)
    p = 1.0 / np.arange(1, E + 1) ** 1.1
    p[[0, 7, E - 1]] = 0
    ids = r.choice(E, size=(M, k), p=p / p.sum()).astype(np.int32)
    al, local = aligned(ids, 0, E, B)
    g, a = bf16((M * k, N), 1), bf16((M * k // top_k, K), 2)
    for dtype, u in ((torch.bfloat16, U16), (torch.float32, U32)):
        dW, db = P.moe_bf16_gemm_wgrad(g.cuda(), a.cuda(), E, *al[:3], top_k, B, bias_grad=True, dtype=dtype)
        for e in range(E):
            s = np.flatnonzero(local == e)
            G, A = g[s].double().numpy(), a[s // top_k].double().numpy()
            want, size = G.T @ A, len(s) * (np.abs(G).T @ np.abs(A))
            assert_close(dW[e], want, ADD * size * (1 + u) + u * np.abs(want) + 1e-30, f"dW[{e}]")
            want, size = G.sum(0), len(s) * np.abs(G).sum(0)
            assert_close(db[e], want, ADD * size * (1 + u) + u * np.abs(want) + 1e-30, f"dbias[{e}]")


@pytest.mark.parametrize("B,expected", [(16, 0), (16, 10000), (32, 0), (128, 0)])
def test_stale_entries_behind_the_live_blocks(B, expected):
    """What stands behind num_tokens_post_padded is not used, whatever it is."""
    M, k, E, N, K = 300, 2, 6, 520, 136
    al, local = aligned(skewed(M, k, E, 3), 0, E, B)
    s, e, n, loc = (t.clone() for t in al)
    live = int(n)
    a, w, g = bf16((M, K), 1).cuda(), bf16((E, N, K), 2).cuda(), bf16((M * k, N), 3).cuda()
    run = lambda s, e: [P.moe_bf16_gemm(a, w, s, e, n, M * k, k, B, expected_slots=expected),  # noqa: E731
                        P.moe_bf16_gemm_dgrad(g, w, s, e, n, loc, k, B, expected_slots=expected),
                        *P.moe_bf16_gemm_wgrad(g, a, E, s, e, n, k, B, bias_grad=True)]
    want = run(al[0], al[1])
    s[live:], e[live // B:] = 5, int(e[live // B - 1])                # a live slot; the last block's expert
    for x, y in zip(run(s, e), want):
        assert torch.equal(x, y)


def big(shape, dtype):
    """Uninitialised device memory of more than 4 GB."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    assert t.numel() * t.element_size() > 2 ** 32
    return t


@pytest.mark.parametrize("B", [16, 32, 128])
def test_rows_beyond_4_gb(B):
    """Activations, outputs and their gradients whose rows lie 1 GB apart."""
    M, E, N, K, ld = 6, 2, 72, 136, 1 << 29
    al, local = aligned(routing(M, 1, E, E, 1), 0, E, B)
    a, w, g = bf16((M, K), 1), bf16((E, N, K), 2), bf16((M, N), 3)
    W = w.cuda()
    A, C, D, X = (big((M, ld), torch.bfloat16) for _ in range(4))
    A[:, :K], D[:, :N] = a.cuda(), g.cuda()
    want = P.moe_bf16_gemm(a.cuda(), W, *al[:3], M, 1, B)
    assert torch.equal(P.moe_bf16_gemm(A[:, :K], W, *al[:3], M, 1, B, out=C[:, :N]), want)
    dA = P.moe_bf16_gemm_dgrad(g.cuda(), W, *al, 1, B)
    assert torch.equal(P.moe_bf16_gemm_dgrad(D[:, :N], W, *al, 1, B, out=X[:, :K]), dA)
    dW, db = P.moe_bf16_gemm_wgrad(g.cuda(), a.cuda(), E, *al[:3], 1, B, bias_grad=True)
    for x, y in zip(P.moe_bf16_gemm_wgrad(D[:, :N], A[:, :K], E, *al[:3], 1, B, bias_grad=True), (dW, db)):
        assert torch.equal(x, y)
    q, s = P.moe_fp8_quant(a.cuda())
    Q = A.view(torch.uint8)[:, :K]
    S = C.view(torch.float32)[:, :2]
    q2, s2 = P.moe_fp8_quant(A[:, :K], out=(X.view(torch.uint8)[:, :K], S))
    assert torch.equal(q2, q.view(torch.uint8)) and torch.equal(s2, s)
    w8, sb = e4m3((E, N, 128), 4).cuda(), scales((E, 1, 1), 4).cuda()
    want = P.moe_w8a8_gemm(q[:, :128].contiguous(), s[:, :1].contiguous(), w8, sb, *al[:3], M, 1, B)
    Q.copy_(q2)
    assert torch.equal(P.moe_w8a8_gemm(Q[:, :128], S[:, :1], w8, sb, *al[:3], M, 1, B, out=D[:, :N]), want)


@pytest.mark.parametrize("B", [16, 32, 128])
def test_weights_beyond_4_gb(B):
    """Experts whose weights, and gradients, start behind 4 GB."""
    E, N, K = 72, 8192, 4096
    ids = torch.tensor([[0], [71], [70], [71]], dtype=torch.int32).numpy()
    al, local = aligned(ids, 0, E, B)
    W = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    normal = lambda *s: torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(2))  # noqa: E731
    w = normal(3, N, K).bfloat16()
    W[0], W[70], W[71] = w[0], w[1], w[2]
    a, g = bf16((4, K), 1).cuda(), bf16((4, N), 3).cuda()
    small, _ = aligned(np.array([[0], [2], [1], [2]], np.int32), 0, 3, B)
    assert torch.equal(P.moe_bf16_gemm(a, W, *al[:3], 4, 1, B, expected_slots=4), P.moe_bf16_gemm(a, w, *small[:3], 4, 1, B))
    assert torch.equal(P.moe_bf16_gemm_dgrad(g, W, *al, 1, B), P.moe_bf16_gemm_dgrad(g, w, *small, 1, B))
    dw, db = P.moe_bf16_gemm_wgrad(g, a, 3, *small[:3], 1, B, bias_grad=True)
    P.moe_bf16_gemm_wgrad(g, a, E, *al[:3], 1, B, bias_grad=True, out=W)
    assert torch.equal(W[0], dw[0]) and torch.equal(W[70], dw[1]) and torch.equal(W[71], dw[2])
    assert not bool(W[1:70].any())
    codes = W.view(torch.uint8).view(2 * E, N, K)                     # 4.8 GB of e4m3
    codes.zero_()
    w8 = (100 * normal(2, N, K)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    sb = scales((2 * E, N // 128, K // 128), 6).cuda()
    codes[1], codes[143] = w8[0], w8[1]
    q, s = P.moe_fp8_quant(a)
    al, _ = aligned(np.array([[1], [143], [143], [1]], np.int32), 0, 2 * E, B)
    small, _ = aligned(np.array([[0], [1], [1], [0]], np.int32), 0, 2, B)
    assert torch.equal(P.moe_w8a8_gemm(q, s, codes, sb, *al[:3], 4, 1, B),
                       P.moe_w8a8_gemm(q, s, w8, sb[[1, 143]].contiguous(), *small[:3], 4, 1, B))


def test_two_streams_at_once():
    M, k, E, N, K, B = 700, 2, 6, 520, 272, 128
    al, _ = aligned(skewed(M, k, E, 1), 0, E, B)
    a, w, g = bf16((M, K), 1).cuda(), bf16((E, N, K), 2).cuda(), bf16((M * k, N), 3).cuda()
    q, s = P.moe_fp8_quant(a)
    w8, sb = e4m3((E, N, K), 4).cuda(), scales((E, -(-N // 128), -(-K // 128)), 4).cuda()

    def run():
        return [P.moe_bf16_gemm(a, w, *al[:3], M * k, k, B, slot_local_ids=al[3]), P.moe_bf16_gemm_dgrad(g, w, *al, k, B),
                *P.moe_bf16_gemm_wgrad(g, a, E, *al[:3], k, B, bias_grad=True),
                P.moe_w8a8_gemm(q, s, w8, sb, *al[:3], M * k, k, B), *P.moe_fp8_quant(a)]

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(run())
    torch.cuda.synchronize()
    for out in got:
        for x, y in zip(out, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("B", [16, 128])
def test_captured_products_follow_the_routing(B):
    """Graphs of the align and the products, replayed with other tokens and other routing; work in one
    caller-owned workspace, eager calls between the replays."""
    M, k, E, N, K = 260, 2, 5, 264, 200
    ids, a, g = torch.zeros((M, k), dtype=torch.int32, device="cuda"), bf16((M, K), 1).cuda(), bf16((M * k, N), 3).cuda()
    w, work = bf16((E, N, K), 2).cuda(), torch.empty(M * k * K, device="cuda")
    w8, sb = e4m3((E, N, K), 4)[:, :, :192].contiguous().cuda(), scales((E, 3, 2), 4).cuda()

    def run(work=None):
        al = P.moe_align(ids, 1, E, B)                                # ids 1 .. E are local
        q, s = P.moe_fp8_quant(a[:, :192].contiguous())
        c8 = torch.zeros((M * k, N), dtype=torch.bfloat16, device="cuda")
        return [P.moe_bf16_gemm(a, w, *al[:3], M * k, k, B, slot_local_ids=al[3]),
                P.moe_bf16_gemm_dgrad(g, w, *al, k, B, work=work),
                *P.moe_bf16_gemm_wgrad(g, a, E, *al[:3], k, B, bias_grad=True),
                P.moe_w8a8_gemm(q, s, w8, sb, *al[:3], M * k, k, B, out=c8)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(work)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = run(work)
    for seed in (1, 2, 3, 4):
        new = routing(M, k, E + 2, E, seed) if seed != 3 else np.full((M, k), 3, np.int32)
        ids.copy_(torch.from_numpy(new))
        a.copy_(bf16((M, K), seed))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, run()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("B,expected", [(16, 0), (16, 1), (16, 10000), (32, 0), (128, 0)])
def test_stale_entries_behind_the_live_blocks_of_the_8_bit_product(B, expected):
    M, k, E, N, K = 300, 2, 6, 520, 272
    al, local = aligned(skewed(M, k, E, 3), 0, E, B)
    s, e, n, _ = (t.clone() for t in al)
    live = int(n)
    a, sa, w, sb = (t.cuda() for t in (e4m3((M, K), 1), scales((M, 3), 1), e4m3((E, N, K), 2), scales((E, 5, 3), 2)))
    run = lambda s, e: P.moe_w8a8_gemm(a, sa, w, sb, s, e, n, M * k, k, B, expected_slots=expected)  # noqa: E731
    want = run(al[0], al[1])
    s[live:], e[live // B:] = 5, int(e[live // B - 1])                # a live slot; the last block's expert
    assert torch.equal(run(s, e), want)
    e[live // B:] = 1 << 30
    assert torch.equal(run(s, e), want)
