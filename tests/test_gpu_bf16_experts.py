"""moe_bf16_gemm, its gradients and moe_experts_linear against 64 bits, and the gradients against
differences."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests.experts_util import ADD, U16, U32, aligned, assert_close, bf16, product, routing, strided

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1, 8, 8, 16), (1, 2, 8, 2048, 512, 16), (5, 8, 16, 136, 72, 16), (53, 2, 6, 264, 200, 7),
          (130, 4, 8, 520, 136, 32), (300, 2, 4, 512, 1024, 64), (513, 4, 8, 392, 264, 128), (640, 1, 3, 128, 576, 128),
          (200, 2, 2, 64, 256, 256), (65, 3, 5, 2880, 96, 100)]


def gradients(dC, A, W, local, top_k):
    """dA, dW, db in 64 bits, with the bound on each before it is stored."""
    dA, SA = np.zeros(A.shape), np.zeros(A.shape)
    dW, SW = np.zeros(W.shape), np.zeros(W.shape)
    db, SB = np.zeros(W.shape[:2]), np.zeros(W.shape[:2])
    for e in range(W.shape[0]):
        s = np.flatnonzero(local == e)
        a, g = A[s // top_k], dC[s]
        y = g @ W[e]
        np.add.at(dA, s // top_k, y)
        np.add.at(SA, s // top_k, np.abs(g) @ np.abs(W[e]))
        dW[e], SW[e] = g.T @ a, len(s) * (np.abs(g).T @ np.abs(a))
        db[e], SB[e] = g.sum(0), len(s) * np.abs(g).sum(0)
    N = W.shape[1]
    return (dA, (N + 8 + top_k) * ADD * SA), (dW, ADD * SW), (db, ADD * SB)


def stored(v, u):
    want, bound = v
    return want, bound * (1 + u) + u * np.abs(want) + 1e-30


@pytest.mark.parametrize("M,k,E,N,K,B", SHAPES)
@pytest.mark.parametrize("gather", [True, False])
def test_product_and_gradients(M, k, E, N, K, B, gather):
    top_k = k if gather else 1
    seed, rows = M + N + K, M if gather else M * k
    ids = routing(M, k, E + 3, E, seed) if E > 1 else np.zeros((M, k), np.int32)
    al, local = aligned(ids, 1 if E > 1 else 0, E, B)                 # a slice: some slots dropped
    a, w, b, g = bf16((rows, K), seed), bf16((E, N, K), seed + 1), bf16((E, N), seed + 2), bf16((M * k, N), seed + 3)
    g[torch.from_numpy(local < 0)] = float("nan")                     # never read
    A64, W64, G64 = (t.double().numpy() for t in (a, w, g))
    want, bound = product(A64, W64, b.double().numpy(), local, top_k)
    out = torch.full((M * k, N), -5.0, dtype=torch.bfloat16, device="cuda")
    A, W, G = strided(a, K + 8), w.cuda(), strided(g, N + 16)
    P.moe_bf16_gemm(A, W, *al[:3], M * k, top_k, B, bias=b.cuda(), out=out)
    dead = torch.from_numpy(local < 0).cuda()
    assert bool((out[dead] == -5.0).all())
    P.moe_bf16_gemm(A, W, *al[:3], M * k, top_k, B, bias=b.cuda(), out=out, slot_local_ids=al[3])
    assert_close(out, want, bound + U16 * np.abs(want) + 1e-30, "C")
    dA, dW, db = gradients(G64, A64, W64, local, top_k)
    got = P.moe_bf16_gemm_dgrad(G, W, *al, top_k, B)
    assert_close(got, *stored(dA, U16), "dA")
    for dtype, u in ((torch.bfloat16, U16), (torch.float32, U32)):
        gw, gb = P.moe_bf16_gemm_wgrad(G, A, E, *al[:3], top_k, B, bias_grad=True, dtype=dtype)
        assert gw.dtype == gb.dtype == dtype
        assert_close(gw, *stored(dW, u), "dW")
        assert_close(gb, *stored(db, u), "dbias")


@pytest.mark.parametrize("B", [16, 128])
def test_empty_experts_and_nothing_local(B):
    for ids, E in ((routing(50, 2, 9, 9, 3, only=[4]), 9), (routing(50, 2, 9, 3, 3, only=[5, 8]), 3)):
        al, local = aligned(ids, 0, E, B)
        a, w, g = bf16((50, 136), 1), bf16((E, 72, 136), 2), bf16((100, 72), 3)
        dA, dW, db = gradients(*(t.double().numpy() for t in (g, a, w)), local, 2)
        assert_close(P.moe_bf16_gemm_dgrad(g.cuda(), w.cuda(), *al, 2, B), *stored(dA, U16), "dA")
        gw, gb = P.moe_bf16_gemm_wgrad(g.cuda(), a.cuda(), E, *al[:3], 2, B, bias_grad=True, dtype=torch.float32)
        assert_close(gw, *stored(dW, U32), "dW")
        assert_close(gb, *stored(db, U32), "dbias")


def test_no_tokens():
    al = P.moe_align(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 0, 4, 16)
    A = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    W = bf16((4, 32, 64), 1).cuda().requires_grad_(True)
    b = bf16((4, 32), 1).cuda().requires_grad_(True)
    out = P.moe_experts_linear(A, W, al, 2, 16, bias=b)
    assert out.shape == (0, 32)
    out.sum().backward()
    assert A.grad.shape == A.shape and not bool(W.grad.any()) and not bool(b.grad.any())


def mlp(x, w13, b13, w2, gw, al, k, B):
    """A training step's expert layer: gate/up, silu and product, down, weighted sum."""
    I = w2.shape[2]
    h = P.moe_experts_linear(x, w13, al, k, B, bias=b13)
    a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    y = P.moe_experts_linear(a, w2, al, 1, B)
    return (y.view(x.shape[0], k, -1).float() * gw[..., None]).sum(1)


@pytest.mark.parametrize("B", [16, 64])
def test_gradients_of_an_expert_layer(B):
    """Every gradient of a two-product layer against the same layer's float64 autograd on the CPU."""
    M, k, E, H, I = 70, 2, 4, 128, 64
    ids = routing(M, k, E + 2, E, 8)                                   # experts E and E + 1 are elsewhere
    al, local = aligned(ids, 0, E, B)
    t = [bf16((M, H), 1), bf16((E, 2 * I, H), 2, H ** -0.5), bf16((E, 2 * I), 3), bf16((E, H, I), 4, I ** -0.5)]
    gw = torch.rand((M, k), generator=torch.Generator().manual_seed(5))
    dev = [v.cuda().requires_grad_(True) for v in t] + [gw.cuda().requires_grad_(True)]
    ref = [v.double().requires_grad_(True) for v in t] + [gw.double().requires_grad_(True)]
    co = bf16((M, H), 6)
    x, w13, b13, w2, g = ref
    total = 0.0
    for s in np.flatnonzero(local >= 0):
        e, r = int(local[s]), int(s) // k
        h = w13[e] @ x[r] + b13[e]
        a = torch.nn.functional.silu(h[:I]) * h[I:]
        total = total + g[r, int(s) % k] * ((w2[e] @ a) * co[r].double()).sum()
    total.backward()
    out = mlp(*dev[:4], dev[4], al, k, B)
    got = torch.autograd.grad((out * co.cuda().float()).sum(), dev)
    # Every intermediate (h, silu, a, y and their gradients) is rounded to bf16, each off by u16 of its
    # size: at most eight such roundings lie on a path from the loss to a gradient.  As a whole (in the
    # 2-norm) a gradient is then off by at most eight u16 of its terms' norm, which the cancellation
    # in a sum of random terms keeps within twice the gradient's own.
    for have, want, name in zip(got, ref, ("x", "w13", "b13", "w2", "weights")):
        off = (have.double().cpu() - want.grad).norm() / want.grad.norm()
        assert off <= 16 * U16, (name, float(off))


def test_gradients_against_differences():
    """d/dt of sum(C * G) along a direction, with operands whose products and sums are exact in fp32
    and whose results are exact in bf16 (small integers), so that the difference is exact too."""
    M, k, E, N, K, B = 40, 2, 3, 16, 24, 16
    ids = routing(M, k, E, E, 12)
    al, _ = aligned(ids, 0, E, B)
    r = np.random.default_rng(13)
    pick = lambda *s: torch.from_numpy(r.integers(-1, 2, s).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    A, W, b, G = pick(M, K), pick(E, N, K), pick(E, N), pick(M * k, N)
    leaves = [t.clone().requires_grad_(True) for t in (A, W, b)]
    grads = torch.autograd.grad(P.moe_experts_linear(leaves[0], leaves[1], al, k, B, bias=leaves[2]), leaves, G)
    value = lambda *t: (P.moe_experts_linear(t[0], t[1], al, k, B, bias=t[2]).double() * G.double()).sum()  # noqa: E731
    for i, t in enumerate((A, W, b)):
        d = pick(*t.shape)
        up, down = [A, W, b], [A, W, b]
        up[i], down[i] = t + d, t - d
        diff = (value(*up) - value(*down)) / 2
        assert float(diff) == float((grads[i].double() * d.double()).sum()), i


def test_needs_input_grad_and_broadcast_gradients():
    M, k, E, N, K, B = 33, 2, 4, 40, 24, 16
    al, _ = aligned(routing(M, k, E, E, 2), 0, E, B)
    A, W = bf16((M, K), 1).cuda(), bf16((E, N, K), 2).cuda().requires_grad_(True)
    out = P.moe_experts_linear(A, W, al, k, B)
    (dW,) = torch.autograd.grad(out.sum(), W)                           # a gradient of stride 0
    ones, _ = P.moe_bf16_gemm_wgrad(torch.ones_like(out), A, E, *al[:3], k, B)
    assert torch.equal(dW, ones)
    A.requires_grad_(True)
    out = P.moe_experts_linear(A, W.detach(), al, k, B)
    g = bf16((N, M * k), 3).cuda().t()                                  # a transposed one
    (dA,) = torch.autograd.grad(out, A, g)
    assert torch.equal(dA, P.moe_bf16_gemm_dgrad(g.contiguous(), W.detach(), *al, k, B))


def test_a_captured_training_step_replays():
    M, k, E, H, I, B = 64, 2, 4, 64, 64, 32
    ids = torch.from_numpy(routing(M, k, E, E, 4)).cuda()
    leaves = [t.cuda().requires_grad_(True) for t in (bf16((M, H), 1), bf16((E, 2 * I, H), 2), bf16((E, 2 * I), 3),
                                                       bf16((E, H, I), 4))]
    gw, co = torch.rand((M, k), device="cuda"), bf16((M, H), 6).cuda()

    def step():
        al = P.moe_align(ids, 0, E, B)
        return torch.autograd.grad(mlp(*leaves, gw, al, k, B).to(torch.bfloat16), leaves, co)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        grads = step()
    for seed in (5, 6, 7):
        with torch.no_grad():
            leaves[0].copy_(bf16((M, H), seed))
            ids.copy_(torch.from_numpy(routing(M, k, E, E, seed)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(grads, step()):
            assert torch.equal(a, b)


def off_alignment(t, lead):
    """t's values, contiguous, `lead` values behind a 16-byte boundary."""
    v = torch.zeros(t.numel() + lead, dtype=t.dtype, device=t.device)[lead:].view(t.shape)
    v.copy_(t)
    assert v.is_contiguous() and v.data_ptr() % 16 == 2 * lead
    return v


@pytest.mark.parametrize("gather", [True, False])
def test_contiguous_gradients_off_16_byte_boundaries(gather):
    """Contiguous gradients that begin between 16-byte boundaries, as the parts of a concatenation's do."""
    M, k, E, N, K, B = 33, 2, 4, 40, 24, 16
    top_k = k if gather else 1
    al, _ = aligned(routing(M, k, E + 1, E, 2), 0, E, B)
    leaves = [t.cuda().requires_grad_(True) for t in (bf16((M * k // top_k, K), 1), bf16((E, N, K), 2), bf16((E, N), 3))]
    g = bf16((M * k, N), 4).cuda()
    out = P.moe_experts_linear(leaves[0], leaves[1], al, top_k, B, bias=leaves[2])
    want = torch.autograd.grad(out, leaves, g, retain_graph=True)
    for lead in (1, 4):
        got = torch.autograd.grad(out, leaves, off_alignment(g, lead), retain_graph=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), lead
    front = torch.zeros(4, dtype=torch.bfloat16, device="cuda")
    joined = torch.cat([front, out.flatten()])
    got = torch.autograd.grad(joined, leaves, torch.cat([front, g.flatten()]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# (N = 8192: 256-row tiles of an expert's columns; the others 128-row ones)
@pytest.mark.parametrize("M,k,E,N,K,B", [(33, 2, 4, 40, 24, 16), (300, 3, 5, 264, 520, 64), (260, 2, 8, 8192, 256, 32),
                                         (1, 1, 1, 8, 8, 16)])
@pytest.mark.parametrize("gather", [True, False])
def test_the_bias_gradient_alone(M, k, E, N, K, B, gather):
    """Frozen weights: the same bits as beside the weights' gradient, which is neither made nor stored."""
    top_k = k if gather else 1
    al, _ = aligned(routing(M, k, E + 1, E, 2), 0, E, B)
    A, W, b = bf16((M * k // top_k, K), 1).cuda(), bf16((E, N, K), 2).cuda(), bf16((E, N), 3).cuda().requires_grad_(True)
    g = bf16((M * k, N), 4).cuda()
    _, want = P.moe_bf16_gemm_wgrad(g, A, E, *al[:3], top_k, B, bias_grad=True)
    out = P.moe_experts_linear(A, W, al, top_k, B, bias=b)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    (got,) = torch.autograd.grad(out, b, g)
    assert torch.equal(got, want)
    assert W.numel() < 4096 or torch.cuda.max_memory_allocated() - before < 2 * W.numel()
    # and with the rows' gradient
    A.requires_grad_(True)
    dA, db = torch.autograd.grad(P.moe_experts_linear(A, W, al, top_k, B, bias=b), (A, b), g)
    assert torch.equal(db, want) and torch.equal(dA, P.moe_bf16_gemm_dgrad(g, W, *al, top_k, B))


def test_the_bias_gradient_alone_of_no_tokens_and_in_a_graph():
    E, N, K, B = 4, 264, 64, 16
    W, b = bf16((E, N, K), 1).cuda(), bf16((E, N), 2).cuda().requires_grad_(True)
    al = P.moe_align(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 0, E, B)
    out = P.moe_experts_linear(torch.zeros((0, K), dtype=torch.bfloat16, device="cuda"), W, al, 2, B, bias=b)
    (db,) = torch.autograd.grad(out, b, torch.zeros_like(out))
    assert db.shape == b.shape and not bool(db.any())
    del out                                                             # (no eager graph of b lives on)
    M = 90
    ids = torch.from_numpy(routing(M, 2, E, E, 3)).cuda()
    A, g = bf16((M, K), 3).cuda(), bf16((2 * M, N), 4).cuda()

    def step():
        return torch.autograd.grad(P.moe_experts_linear(A, W, P.moe_align(ids, 0, E, B), 2, B, bias=b), b, g)[0]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for seed in (5, 6, 7):
        g.copy_(bf16((2 * M, N), seed))
        ids.copy_(torch.from_numpy(routing(M, 2, E, E, seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, step())
