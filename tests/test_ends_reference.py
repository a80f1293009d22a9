"""The plain 64-bit forms of the router's and the combine's gradients against differences of their
forward forms, and the refusals of the entry points (validated on the host, with addresses that are never used)."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from quantized_mixture_experts_align_amd import _lib as L
from tests import ends_util as U

H = 2.0 ** -14   # step of the central differences: off by about h^2 times third derivatives, and 2^-53 / h


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("part", ["weights", "means", "balance", "all"])
def test_router_gradient_against_differences(score, renorm, part):
    r = np.random.default_rng(5)
    M, E, k, scale = 7, 9, 3, 1.7
    l = 1.5 * r.standard_normal((M, E))
    l[2, 4] = l[3, :7] = -np.inf                      # row 3 has two experts for three choices
    live = np.array([0, 3, 0, 0, -1, 0, 0])
    ids = U.choose64(l, score, 0.1 * r.standard_normal(E), k, live)
    assert ids[3, 2] == -1 and (ids[4] == -1).all()
    dw = r.standard_normal((M, k)) if part in ("weights", "all") else None
    dm = r.standard_normal(E) if part in ("means", "all") else None
    db = 0.7 if part in ("balance", "all") else None
    counts = U.router64(l, score, ids, renorm, scale, live)[1]

    def value(l):
        w, _, means, _, _ = U.router64(l, score, ids, renorm, scale, live)
        v = 0.0 if dw is None else (dw * w).sum()
        v += 0.0 if dm is None else (dm * means).sum()
        return v + (0.0 if db is None else db * E * (counts * means).sum() / counts.sum())

    got, mag = U.router_grad64(l, score, ids, renorm, scale, live, dw, dm, db)
    assert (np.abs(got) <= mag * (1 + 1e-12) + 1e-300).all()
    for t in range(M):
        for e in range(E):
            if np.isneginf(l[t, e]):
                assert got[t, e] == 0.0
                continue
            up, down = l.copy(), l.copy()
            up[t, e] += H
            down[t, e] -= H
            assert abs((value(up) - value(down)) / (2 * H) - got[t, e]) < 1e-7, (t, e)


@pytest.mark.parametrize("norm", [False, True])
def test_combine_gradient_against_differences(norm):
    r = np.random.default_rng(6)
    M, k, W, eps, c = 3, 2, 8, 1e-3, 1.4
    y, g, dout = r.standard_normal((M, k, W)), r.standard_normal((M, k)), r.standard_normal((M, W))
    live = np.array([[True, True], [False, True], [False, False]])
    n = 1.0 + 0.3 * r.standard_normal(W) if norm else None
    _, dy, dg, dn = U.combine64(y, g, live, n, eps, c, dout)[:4]
    value = lambda y, g, n: (U.combine64(y, g, live, n, eps, c, dout)[0] * dout).sum()  # noqa: E731

    def slope(at, v):
        up, down = v.copy(), v.copy()
        up[at] += H
        down[at] -= H
        return up, down

    for at in np.ndindex(y.shape):
        up, down = slope(at, y)
        assert abs((value(up, g, n) - value(down, g, n)) / (2 * H) - dy.reshape(M, k, W)[at]) < 1e-6
    for at in np.ndindex(g.shape):
        up, down = slope(at, g)
        assert abs((value(y, up, n) - value(y, down, n)) / (2 * H) - dg[at]) < 1e-6
    if norm:
        for at in np.ndindex(n.shape):
            up, down = slope(at, n)
            assert abs((value(y, g, up) - value(y, g, down)) / (2 * H) - dn[at]) < 1e-6


A16 = 0x10000          # an aligned address
ROUTER = dict(logits=A16, f32=0, ld=64, M=4, E=64, bias=None, live=None, score=0, top_k=4, renorm=1, scale=1.0, ids=A16,
              weights=A16, counts=None, means=None, balance=None, tokens=None, work=None, work_bytes=0, stream=None)
STATS = dict(counts=A16, means=A16, balance=A16, tokens=A16, work=A16, work_bytes=1 << 20)
GRAD = dict(logits=A16, f32=0, ld=64, M=4, E=64, live=None, score=0, top_k=4, renorm=1, scale=1.0, ids=A16, dw=A16,
            counts=A16, tokens=A16, d_means=None, d_balance=A16, dx=A16, ld_d=64, stream=None)
COMBINE = dict(y=A16, w=A16, local=A16, norm=A16, eps=1e-6, rsf=1.0, M=4, top_k=2, H=64, dout=A16, ld=64, dy=A16, dw=A16,
               dn=A16, work=A16, elems=4 * 64, stream=None)
ADAPT = dict(base=A16, ldb=128, x=A16, x_rows=16, ldx=256, A=A16, B=A16, scales=None, ranks=None, L=4, r=16, N=128, K=256,
             out=A16, ldo=128, sorted=A16, eids=A16, ntpp=A16, live=A16, numel=16, top_k=1, block_m=16, work=A16,
             elems=1 << 20, stream=None)
FAR = A16 + (1 << 24)

BAD = [
    ("moe_router", ROUTER, L.MOE_EINVAL, [dict(logits=None), dict(ids=None), dict(weights=None), dict(M=-1), dict(E=0),
                                          dict(top_k=0), dict(top_k=65), dict(ld=63), dict(score=2), dict(score=-1),
                                          dict(counts=A16), {**STATS, "means": None}, {**STATS, "work": None},
                                          {**STATS, "tokens": None}]),
    ("moe_router", ROUTER, L.MOE_EUNSUPPORTED, [dict(E=1025, ld=1025), dict(top_k=17), dict(M=(1 << 25) + 1), dict(logits=A16 + 1),
                                                dict(logits=A16 + 2, f32=1), dict(ids=A16 + 2), dict(weights=A16 + 2),
                                                dict(bias=A16 + 2), dict(live=A16 + 2), {**STATS, "work": A16 + 4}]),
    ("moe_router", ROUTER, L.MOE_ESIZE, [{**STATS, "work_bytes": 16 + 8 * 64 + 3}]),
    ("moe_router_grad", GRAD, L.MOE_EINVAL, [dict(logits=None), dict(dx=None), dict(ids=None), dict(counts=None),
                                             dict(tokens=None), dict(ld_d=63), dict(ld=60), dict(score=5), dict(top_k=0)]),
    ("moe_router_grad", GRAD, L.MOE_EUNSUPPORTED, [dict(dx=A16 + 1), dict(dx=A16 + 2, f32=1), dict(dw=A16 + 1),
                                                   dict(d_balance=A16 + 2), dict(E=2000, ld=2000, ld_d=2000)]),
    ("moe_combine_grad", COMBINE, L.MOE_EINVAL, [dict(y=None), dict(w=None), dict(local=None), dict(dout=None), dict(ld=56),
                                                 dict(norm=None), dict(dy=None, dw=None, dn=None)]),
    ("moe_combine_grad", COMBINE, L.MOE_EUNSUPPORTED, [dict(H=60), dict(H=0), dict(top_k=0), dict(top_k=17), dict(M=-1), dict(M=1 << 24),
                                                       dict(ld=68), dict(y=A16 + 8), dict(dout=A16 + 8), dict(dy=A16 + 8),
                                                       dict(norm=A16 + 8), dict(dn=A16 + 1), dict(work=A16 + 8)]),
    ("moe_combine_grad", COMBINE, L.MOE_ESIZE, [dict(elems=4 * 64 - 1), dict(work=None)]),
    ("moe_adapters_add", ADAPT, L.MOE_EINVAL, [dict(base=None), dict(x=None), dict(A=None), dict(B=None), dict(out=None),
                                               dict(sorted=None), dict(eids=None), dict(ntpp=None), dict(work=None),
                                               dict(out=FAR, live=None), dict(out=A16 + 16), dict(ldo=136), dict(L=0), dict(r=0),
                                               dict(N=0), dict(K=0), dict(numel=-1), dict(top_k=0), dict(block_m=0),
                                               dict(block_m=257), dict(x_rows=15), dict(ldx=248), dict(ldb=120, ldo=120)]),
    ("moe_adapters_add", ADAPT, L.MOE_EUNSUPPORTED, [dict(r=12), dict(r=264), dict(N=124), dict(K=252), dict(L=513), dict(ldx=260),
                                                     dict(x=A16 + 8), dict(base=A16 + 8, out=A16 + 8), dict(A=A16 + 8),
                                                     dict(B=A16 + 8), dict(work=A16 + 8), dict(scales=A16 + 2),
                                                     dict(ranks=A16 + 2), dict(numel=1 << 31, x_rows=1 << 31)]),
    ("moe_adapters_add", ADAPT, L.MOE_ESIZE, [dict(elems=16 * 16 - 1)]),
]


@pytest.mark.parametrize("name,good,code,changes", BAD, ids=[f"{b[0]}-{-b[2]}" for b in BAD])
def test_entry_points_refuse(name, good, code, changes):
    f = getattr(L.lib(), name)
    for change in changes:
        args = {**good, **change}
        assert list(args) == list(good)
        assert f(*args.values()) == code, change
        assert name.encode() in L.lib().moe_last_error(), change


def test_empty_batches_launch_nothing():
    for name, good, change in (("moe_router", ROUTER, dict(M=0, logits=None, ids=None, weights=None)),
                               ("moe_router_grad", GRAD, dict(M=0, logits=None, dx=None, ids=None, dw=None)),
                               ("moe_combine_grad", COMBINE, dict(M=0, y=None, w=None, local=None, dout=None, dy=None, dw=None,
                                                                  norm=None, dn=None)),
                               ("moe_adapters_add", ADAPT, dict(numel=0, base=None, x=None, out=None, work=None))):
        assert getattr(L.lib(), name)(*{**good, **change}.values()) == L.MOE_OK, name


def test_workspace_sizes():
    # statistics: the totals, and for each of at most 256 workgroups of 32 tokens (8 above 512 experts) E sums and counts
    # and its tokens
    assert P.router_workspace(1, 8) == 16 + 8 * 8 + 4
    assert P.router_workspace(65, 256) == 16 + 3 * (8 * 256 + 4)
    assert P.router_workspace(1 << 20, 1024) == 16 + 256 * (8 * 1024 + 4)
    assert P.router_workspace(0, 8) == P.router_workspace(1, 8)
    # the inner products of every row, times at most 32 for short batches
    for numel, n, r, K, B in ((1, 8, 16, 7168, 16), (64, 64, 16, 4096, 16), (8179, 6, 64, 4096, 64), (5, 1, 256, 8, 1)):
        e = P.adapters_workspace(numel, n, r, K, B)
        assert e % (numel * r) == 0 and 1 <= e // (numel * r) <= 32
    assert P.adapters_workspace(0, 8, 16, 64, 16) == 0
    for call in (lambda: P.router_workspace(-1, 8), lambda: P.router_workspace(1, 1025), lambda: P.combine_grad_workspace(-1, 8),
                 lambda: P.adapters_workspace(1, 8, 12, 64, 16)):
        with pytest.raises(ValueError):
            call()


def test_host_tensors_and_unknown_names_are_refused():
    x, i = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((4, 1), dtype=torch.int32)
    w, a = torch.zeros((4, 1)), torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    for call in (lambda: P.moe_router(x, 2), lambda: P.moe_experts_router(x, 2), lambda: P.moe_router_grad(x, i),
                 lambda: P.moe_combine_grad(x, w, i, x), lambda: P.moe_experts_combine(x, w, i),
                 lambda: P.moe_adapters_add(x, x, a, a, (i, i, i, i), 16)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    for call in (lambda: P.moe_router(x, 2, score="relu"), lambda: P.moe_experts_router(x, 2, score=""),
                 lambda: P.moe_router_grad(x, i, score="top")):
        with pytest.raises(ValueError, match="unknown score"):
            call()
