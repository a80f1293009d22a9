"""Plain 64-bit forms and error bounds of the products with 8-bit and bf16 expert weights.

The bounds count roundings: u16 = 2^-8 for a value stored as bf16, u32 = 2^-24 for one stored in
fp32, and 2^-23 of the sum of the terms' magnitudes for each term added in fp32 (one unit in the
last place, so that an accumulator which cuts instead of rounding is covered too)."""
import numpy as np
import torch

U16, U32, ADD = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23
BLOCK = 128


def routing(M, k, E_all, E, seed, only=None):
    """topk_ids int32 [M, k] over E_all experts (distinct per token); `only`: ids drawn from these."""
    r = np.random.default_rng([seed, 77])
    pool = np.arange(E_all) if only is None else np.asarray(only)
    return np.stack([r.choice(pool, size=k, replace=len(pool) < k) for _ in range(M)]).astype(np.int32).reshape(M, k)


def aligned(ids, start, E, B):
    """(device align outputs, slot -> local expert or -1 as numpy)."""
    import quantized_mixture_experts_align_amd as P
    al = P.moe_align(torch.from_numpy(ids).cuda(), start, E, B)
    local = np.where((ids >= start) & (ids < start + E), ids - start, -1).reshape(-1)
    return al, local


def bf16(shape, seed, scale=1.0):
    r = np.random.default_rng([seed, 78])
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


def e4m3(shape, seed):
    r = np.random.default_rng([seed, 79])
    return torch.from_numpy((r.standard_normal(shape) * 100).clip(-448, 448).astype(np.float32)).to(torch.float8_e4m3fn)


def scales(shape, seed):
    r = np.random.default_rng([seed, 80])
    return torch.from_numpy(np.exp(r.normal(-5.0, 1.0, shape)).astype(np.float32))


def spread(s, N, K):
    """Scales [.., ceil(N/128) or N, ceil(K/128)] over [.., N, K] (float64)."""
    s = np.repeat(s.double().numpy(), BLOCK, axis=-1)[..., :K]
    return s if s.shape[-2] == N else np.repeat(s, BLOCK, axis=-2)[..., :N, :]


def product(A, W, bias, local, top_k):
    """(C [numel, N], bound on its error before it is stored, without the storing) for float64 A
    [rows, K] and W [E, N, K]; rows of dropped slots are zero."""
    numel, N, K = len(local), W.shape[1], A.shape[1]
    C, S = np.zeros((numel, N)), np.zeros((numel, N))
    for e in range(W.shape[0]):
        s = np.flatnonzero(local == e)
        a = A[s // top_k]
        C[s], S[s] = a @ W[e].T, np.abs(a) @ np.abs(W[e]).T
        if bias is not None:
            C[s] += bias[e]
            S[s] += np.abs(bias[e])
    return C, (K + 8) * ADD * S


def product8(a, sa, w, sb, bias, local, top_k):
    """`product` of e4m3fn operands with their scales, and the bound for their matrix instruction.

    That instruction adds the products of eight consecutive k on the exponent of the largest, cut 13
    places below it (2^16 + 2^3 keeps its small term, 2^16 + 2^2 does not; a product of another eight
    is added in full fp32: checked on the card with single products).  Of eight products, seven can
    lose up to 2^-13 of the largest each, so a group is off by at most 7 * 2^-13 * max |p|, and
    max |p| is at most the root of the sum of the squares."""
    rows, K = a.shape
    N = w.shape[1]
    A, W = a.double().numpy() * spread(sa, rows, K), w.double().numpy() * spread(sb, N, K)
    C, bound = product(A, W, bias, local, top_k)
    for e in range(W.shape[0]):
        s = np.flatnonzero(local == e)
        a2, w2 = A[s // top_k] ** 2, W[e].T ** 2
        for k in range(0, K, 8):
            bound[s] += 7 * 2.0 ** -13 * np.sqrt(a2[:, k: k + 8] @ w2[k: k + 8])
    return C, bound


def assert_close(got, want, bound, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want)
    bad = np.argwhere(~(off <= bound))
    assert bad.size == 0, (f"{what}: {len(bad)} of {got.size} outside their bound; at {tuple(bad[0])}: got "
                           f"{got[tuple(bad[0])]:.8g} want {want[tuple(bad[0])]:.8g} bound {bound[tuple(bad[0])]:.3g}")


def strided(t, ld, fill=float("nan")):
    """t [R, C] as a view into device rows of `ld` values, the rest of each row filled."""
    base = torch.full((t.shape[0], ld), fill, dtype=torch.float32).to(t.dtype).cuda()
    base[:, : t.shape[1]] = t.cuda()
    return base[:, : t.shape[1]]
