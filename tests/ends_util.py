"""Plain 64-bit forms of the operators at the experts' two ends -- the router with its statistics and
gradients, the combine's gradients, adapters -- and bounds on the errors of fp32 forms of them.

The bounds count roundings as tests/experts_util.py does (U16, U32 for a stored value, ADD for each term added in
fp32).  An exponential in fp32 is off by EXP = 4 ADD of its value (the hardware's exp2 by one unit, the product with
log2 e, the correction of it and a reciprocal by less than one each) and by U32 for each unit of its argument,
whose own rounding enters as a relative error."""
import numpy as np
import torch

from tests.experts_util import ADD, U16, U32

EXP = 4 * ADD


def softmax64(l):
    top = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
    s = e.sum(1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def log_sigmoid64(l):
    return np.where(l >= 0, -np.log1p(np.exp(-np.abs(l))), l - np.log1p(np.exp(-np.abs(l))))


def normed_sigmoid64(l):
    """sigmoids over their sum in a row (0 in a row without any), exact however small they are"""
    return softmax64(log_sigmoid64(l))


def choose64(l, score, bias, k, live):
    """ids [M, k] of a row's largest logits, or scores + bias; -1 where nothing is left."""
    M, E = l.shape
    key = l if bias is None else (softmax64(l) if score == "softmax" else np.exp(log_sigmoid64(l))) + bias
    key = np.where((l > -np.inf) & (np.ones(E) if bias is None else bias > -np.inf).astype(bool), key, -np.inf)
    ids = np.full((M, k), -1, np.int32)
    for t in range(M):
        if live is None or live[t] >= 0:
            order = sorted((e for e in range(E) if key[t, e] > -np.inf), key=lambda e: (-key[t, e], e))[:k]
            ids[t, : len(order)] = order
    return ids


def router64(l, score, ids, renorm, scale, live):
    """(weights, counts, means, balance, tokens) for logits l (float64 [M, E], no NaN) and the chosen ids."""
    M, E = l.shape
    has, at = ids >= 0, np.maximum(ids, 0)
    x = np.where(has, np.take_along_axis(l, at, 1), -np.inf)
    if renorm:
        w = softmax64(x) if score == "softmax" else normed_sigmoid64(x)
    else:
        w = np.take_along_axis(softmax64(l) if score == "softmax" else np.exp(log_sigmoid64(l)), at, 1)
    on = np.ones(M, bool) if live is None else live >= 0
    q = softmax64(l) if score == "softmax" else normed_sigmoid64(l)
    counts = np.bincount(ids[has], minlength=E)
    tokens = int(on.sum())
    means = q[on].sum(0) / max(tokens, 1)
    return scale * np.where(has, w, 0.0), counts, means, E * (counts * means).sum() / max(counts.sum(), 1), tokens


def router_grad64(l, score, ids, renorm, scale, live, dw, d_means, d_balance):
    """(gradient, the sum of the magnitudes of the terms of each of its values) of
    sum dw * weights + sum d_means * means + d_balance * balance with the counts held constant."""
    M, E = l.shape
    _, counts, _, _, tokens = router64(l, score, ids, renorm, scale, live)
    has, at = ids >= 0, np.maximum(ids, 0)
    g, mag = np.zeros((M, E)), np.zeros((M, E))
    q = softmax64(l) if score == "softmax" else normed_sigmoid64(l)
    other = np.exp(log_sigmoid64(-l)) if score == "sigmoid" else np.ones((M, E))      # 1 - s
    if dw is not None:
        h = router64(l, score, ids, renorm, 1.0, live)[0]
        slope = np.take_along_axis(other, at, 1)
        dot, size = (dw * h).sum(1, keepdims=True), (np.abs(dw) * h).sum(1, keepdims=True)
        d = scale * h * slope * (dw - dot * renorm)
        m = abs(scale) * h * slope * (np.abs(dw) + size * renorm)
        for j in range(ids.shape[1]):
            r = np.flatnonzero(has[:, j])
            g[r, ids[r, j]] += d[r, j]
            mag[r, ids[r, j]] += m[r, j]
        if score == "softmax" and not renorm:
            g -= scale * q * dot
            mag += abs(scale) * q * size
    a = np.zeros(E) if d_means is None else d_means.copy()
    if d_balance is not None:
        a += d_balance * E * counts / max(counts.sum(), 1)
    a /= max(tokens, 1)
    g += q * other * (a - (q * a).sum(1, keepdims=True))
    mag += q * other * (np.abs(a) + (q * np.abs(a)).sum(1, keepdims=True))
    if live is not None:
        g[live < 0] = mag[live < 0] = 0.0
    return g, mag


def router_error(l, E):
    """Relative error of a sum of exponentials, of their ratios and of what is made of a few of them: EXP for
    each of four factors, U32 for each unit of the arguments' differences, ADD for the up to 16 terms a lane adds,
    six exchanges, and a dozen products."""
    finite = l[np.isfinite(l)]
    spread = 2 * np.abs(np.clip(finite, -110.0, 110.0)).max() if finite.size else 0.0
    return 4 * EXP + 2 * spread * U32 + (16 + 6 + 12) * ADD


def combine64(y, g, live, n, eps, c, dout):
    """(out, dy, dg, dn) and bounds of the last three without the storing; y [M, k, H], g [M, k], live [M, k]."""
    M, k, H = y.shape
    y = np.where(live[..., None], y, 0.0)
    g = g * live
    z = y * (1.0 if n is None else n)
    r = np.ones((M, k)) if n is None else 1.0 / np.sqrt((z * z).mean(2) + eps)
    out = c * ((g * r)[..., None] * z).sum(1)
    d, size = (dout[:, None] * z).sum(2), (np.abs(dout)[:, None] * np.abs(z)).sum(2)
    # a sum of H products: eight a lane and chunk, the chunks, the exchanges; r: the sum, a quotient, a root
    adds = (H + 16) * ADD
    dg, dg_b = c * r * d * live, abs(c) * r * size * live * (2 * adds + 8 * ADD)
    f = (c * g * r)[..., None]
    if n is None:
        dz, dz_b = f * dout[:, None], np.abs(f * dout[:, None]) * 4 * ADD
    else:
        back = (r * r * d / H)[..., None] * z
        dz = f * (dout[:, None] - back)
        dz_b = np.abs(f) * ((np.abs(dout[:, None]) + np.abs(back)) * (2 * adds + 16 * ADD) +
                            (r * r * size / H)[..., None] * np.abs(z) * adds)
    m = 1.0 if n is None else n
    dy, dy_b = dz * m, dz_b * np.abs(m) * (1 + ADD) + np.abs(dz * m) * ADD
    dn = (dz * y).sum((0, 1))
    dn_b = (dz_b * np.abs(y)).sum((0, 1)) + (np.abs(dz * y)).sum((0, 1)) * (M * k + 16) * ADD
    return out, dy.reshape(M * k, H), dg, dn, dy_b.reshape(M * k, H), dg_b, dn_b


def adapters64(base, x, A, B, scales, ranks, ids, top_k):
    """(out, its bound without the storing) for float64 operands; ids [numel], -1 without an adapter."""
    out, bound = base.copy(), np.zeros_like(base)
    K = x.shape[1]
    for a in range(A.shape[0]):
        m = np.flatnonzero(ids == a)
        r = A.shape[1] if ranks is None else min(max(int(ranks[a]), 0), A.shape[1])
        if not len(m) or not r:
            continue
        s = 1.0 if scales is None else scales[a]
        xr, Ar, Br = x[m // top_k], A[a, :r], B[a, :, :r]
        t, size = s * (xr @ Ar.T), abs(s) * (np.abs(xr) @ np.abs(Ar).T)
        out[m] += t @ Br.T
        # the inner sums, their two halves (2^-8 of 2^-8), the outer sums of twice r terms
        terms = np.abs(t) @ np.abs(Br).T
        bound[m] = size @ np.abs(Br).T * (K + 40) * ADD * (1 + U16) + terms * (U16 * U16 + (2 * r + 24) * ADD)
    return out, bound + 2 * ADD * np.abs(out) + np.abs(base) * ADD


def np64(t):
    return t.detach().double().cpu().numpy()


def logits(M, E, dtype, seed, spread=2.0):
    r = np.random.default_rng([seed, 81])
    return torch.from_numpy((spread * r.standard_normal((M, E))).astype(np.float32)).to(dtype)
