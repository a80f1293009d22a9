"""The router with its counts, balance loss and gradients against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests import ends_util as U
from tests.experts_util import ADD, U16, U32, assert_close, strided
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(lg, k, score, bias, renorm, scale, live, dw, d_means, d_balance, what):
    """Every output and gradient of one batch (lg: device logits, the rest numpy or None)."""
    l, (M, E) = U.np64(lg), lg.shape
    dev = lambda a, t=F32: None if a is None else torch.from_numpy(np.asarray(a)).to(t).cuda()  # noqa: E731
    how = dict(score=score, renormalise=renorm, scale=scale, live=dev(live, torch.int32))
    announce(what)
    ids, w, st = P.moe_router(lg, k, bias=dev(bias), stats=True, **how)
    want = U.choose64(l, score, bias, k, live)
    assert (ids.cpu().numpy() == want).all(), (what, np.argwhere(ids.cpu().numpy() != want)[:3])
    w64, counts, means, balance, tokens = U.router64(l, score, want, renorm, scale, live)
    err = U.router_error(l, E)
    tiny = 2.0 ** -125
    assert_close(w, w64, err * np.abs(w64) + abs(scale) * tiny, what + " weights")
    assert (st.counts.cpu().numpy() == counts).all() and int(st.tokens) == tokens
    per_lane = -(-M // 4096) + 4     # a lane's tokens, then the workgroups' sums in 64 bits
    assert_close(st.means, means, (err + per_lane * ADD) * means + tiny, what + " means")
    assert_close(st.balance, np.array([balance]), np.array([(err + per_lane * ADD) * balance + tiny]), what + " balance")
    alone = P.moe_router(lg, k, bias=dev(bias), **how)
    assert torch.equal(alone[0], ids) and torch.equal(alone[1], w)
    g64, mag = U.router_grad64(l, score, want, renorm, scale, live, dw, d_means, d_balance)
    got = P.moe_router_grad(lg, ids, dev(dw), stats=st, d_means=dev(d_means), d_balance=None if d_balance is None else
                            torch.tensor([d_balance], device="cuda"), **how)
    store = U16 if lg.dtype is BF else U32
    # (the coefficients of the loss: an E-fold count ratio, a product, a sum and a quotient)
    limit = (2 * err + (E // 16 + 8 + 16) * ADD) * mag
    assert_close(got, g64, limit * (1 + store) + store * np.abs(g64) + tiny, what + " gradient")


SIZES = [(1, 1, 1), (5, 3, 3), (33, 8, 2), (17, 16, 16), (4, 60, 6), (67, 64, 8), (9, 65, 4), (66, 128, 4), (130, 129, 5),
         (1, 256, 8), (257, 256, 8), (7, 257, 8), (35, 384, 6), (64, 512, 10), (3, 513, 16), (37, 1000, 7), (21, 1024, 16)]


@pytest.mark.parametrize("M,E,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_statistics_and_gradient(M, E, k, dtype, score):
    r = np.random.default_rng([M, E, k])
    lg = U.logits(M, E, dtype, M + E).cuda()
    for bias in (None, (0.2 * r.standard_normal(E)).astype(np.float32)):
        for renorm in (False, True):
            check(lg, k, score, bias, renorm, 1.0 if renorm else 2.5, None, r.standard_normal((M, k)).astype(np.float32),
                  r.standard_normal(E).astype(np.float32), 0.37, f"M={M} E={E} k={k} {dtype} {score} {bias is not None} {renorm}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_masks_padding_and_too_few_experts(dtype, score, biased):
    r = np.random.default_rng(3)
    M, E, k = 70, 40, 6
    lg = U.logits(M, E, dtype, 9)
    lg[:, 5] = -float("inf")                       # an expert that is switched off
    lg[3, 2:] = -float("inf")                      # fewer experts than choices
    lg[4] = -float("inf")                          # none
    live = np.where(r.random(M) < 0.3, -1, r.integers(0, 5, M)).astype(np.int32)
    live[3] = live[4] = 0
    bias = (0.1 * r.standard_normal(E)).astype(np.float32) if biased else None
    if biased:
        bias[7] = -np.inf
    for renorm in (False, True):
        check(lg.cuda(), k, score, bias, renorm, 1.3, live, r.standard_normal((M, k)).astype(np.float32), None, 1.0,
              f"masks {dtype} {score} {biased} {renorm}")
    gone = np.full(M, -1, np.int32)                # a batch of padding: nothing counts
    ids, w, st = P.moe_router(lg.cuda(), k, score=score, live=torch.from_numpy(gone).cuda(), stats=True)
    assert int(ids.max()) == -1 and float(w.abs().max()) == 0 and int(st.counts.abs().max()) == 0
    assert float(st.balance) == 0.0 and float(st.means.abs().max()) == 0 and int(st.tokens) == 0
    got = P.moe_router_grad(lg.cuda(), ids, torch.ones_like(w), score=score, live=torch.from_numpy(gone).cuda(), stats=st,
                            d_balance=torch.ones(1, device="cuda"))
    assert float(got.abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E", [12, 256, 700])
def test_ties_fall_to_the_lower_index(dtype, biased, E):
    r = np.random.default_rng(E)
    lg = torch.from_numpy(r.integers(-1, 2, (33, E)).astype(np.float32)).to(dtype)
    lg[0] = 0.0
    lg[1, ::2] = -0.0                              # equal to +0
    lg[1, 1::2] = 0.0
    bias = np.zeros(E, np.float32) if biased else None
    for score in ("softmax", "sigmoid"):
        check(lg.cuda(), 8, score, bias, True, 1.0, None, r.standard_normal((33, 8)).astype(np.float32), None, None, f"ties {score}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biased_scores_that_differ_in_the_tenth_place(score):
    """Selection keys 2^-30 apart: equal in fp32, told apart in 64 bits."""
    M, E, k = 32, 64, 8
    r = np.random.default_rng(8)
    l = np.zeros((M, E), np.float32)
    for t in range(M):
        l[t] = r.permutation(E) * 2.0 ** (-30 if score == "sigmoid" else -24)
    bias = np.full(E, 0.5, np.float32)
    got = P.moe_router(torch.from_numpy(l).cuda(), k, score=score, bias=torch.from_numpy(bias).cuda())[0]
    assert (got.cpu().numpy() == U.choose64(l.astype(np.float64), score, bias, k, None)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score,bias,low,high", [
    ("sigmoid", 0.0, 30.0, 33.0), ("sigmoid", 0.0, 31.0, 36.0), ("sigmoid", 0.0, 30.0, 31.0), ("sigmoid", 0.0, 28.0, 28.125),
    ("sigmoid", 1.0, -30.0, -29.5), ("sigmoid", -1.0, 30.0, 33.0), ("softmax", 1.0, -30.5, -30.0), ("softmax", 0.5, -31.0, -30.0)])
@pytest.mark.parametrize("E,k", [(24, 3), (256, 8), (256, 12), (700, 16)])
def test_biased_scores_that_differ_in_the_last_places(score, bias, low, high, dtype, E, k):
    """Scores 2^-43 to 2^-50 apart, the larger at the higher index, at the last place of the choice."""
    l = np.full((5, E), -60.0 if bias > 0 else -6.0, np.float32)
    for t in range(5):
        l[t, t + 1: t + k] = 0.0 if score == "softmax" else 36.0 - low if low < 0 else 60.0
        l[t, t + k + 1], l[t, E - 1 - t] = low, high
    lg, b = torch.from_numpy(l).to(dtype).cuda(), np.full(E, bias, np.float32)
    want = U.choose64(U.np64(lg), score, b, k, None)
    assert (want[:, -1] == E - 1 - np.arange(5)).all()
    got = P.moe_router(lg, k, score=score, bias=torch.from_numpy(b).cuda())[0]
    assert (got.cpu().numpy() == want).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,k", [(24, 8), (129, 8), (256, 8), (256, 12), (700, 8), (1000, 16)])
@pytest.mark.parametrize("bias", [0.0, 1.0])
def test_biased_choice_of_saturated_scores(dtype, E, k, bias):
    """Sigmoids within e^-15 of 1, or of 0 beside a bias of 1, from logits 1/8 apart, many of them equal.  At |x| = 33 a step of
    1/8 moves the score by 6.2e-16; a sum with 1, a quotient and their counterparts in the 64-bit form are off by
    2^-53 (1.1e-16) each at most, so the order is the same in both."""
    r = np.random.default_rng([E, k])
    l = r.integers(120, 265, (33, E)) / 8.0 * (1.0 if bias == 0.0 else -1.0)
    lg, b = torch.from_numpy(l.astype(np.float32)).to(dtype).cuda(), np.full(E, bias, np.float32)
    got = P.moe_router(lg, k, score="sigmoid", bias=torch.from_numpy(b).cuda())[0]
    assert (got.cpu().numpy() == U.choose64(U.np64(lg), "sigmoid", b, k, None)).all()


def near_ties(M, E, top, score, biased, seed):
    """Logits (fp32) and biases whose `top` best experts of a row lie within a few 2^-24 of each other (their order is
    another in every row), the others well below."""
    r = np.random.default_rng([seed, E])
    close = r.permutation(top) * 1.0
    order = np.stack([r.permutation(E) for _ in range(M)])
    l = np.full((M, E), -6.0) + 0.5 * r.standard_normal((M, E))
    bias = (0.05 * r.random(E)).astype(np.float32) if biased else None
    for t in range(M):
        e = order[t, :top]
        delta = r.permutation(close) * 2.0 ** -23
        if not biased:
            l[t, e] = 2.0 + delta
        elif score == "sigmoid":
            s = 0.8 - bias[e] + delta
            l[t, e] = np.log(s / (1.0 - s))
        else:                                      # probabilities of about 0.6 / top, what is left for the others
            p = 0.6 / top * (1.05 - bias[e]) + delta
            l[t, e] = np.log(p)
            rest = np.setdiff1d(np.arange(E), e)
            l[t, rest] += np.log((1.0 - p.sum()) / np.exp(l[t, rest]).sum())
    if biased and score == "softmax":
        bias = (bias * np.float32(0.6 / top)).astype(np.float32)
    return l.astype(np.float32), bias


@pytest.mark.parametrize("E,top,k", [(24, 6, 4), (64, 12, 8), (129, 5, 3), (256, 14, 8), (512, 12, 7), (1000, 30, 8), (256, 40, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_near_ties_are_ordered_exactly(E, top, k, score, biased):
    """A few candidates of a row closer than fp32 keys tell apart, and more of them than a group has lanes."""
    l, bias = near_ties(37, E, top, score, biased, k)
    got = P.moe_router(torch.from_numpy(l).cuda(), k, score=score, renormalise=True,
                       bias=None if bias is None else torch.from_numpy(bias).cuda())
    want = U.choose64(l.astype(np.float64), score, bias, k, None)
    assert (got[0].cpu().numpy() == want).all()
    w = U.router64(l.astype(np.float64), score, want, True, 1.0, None)[0]
    assert_close(got[1], w, U.router_error(l, E) * w, "weights")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("at", [-1e30, -3e4, -150.0, 80.0, 1e30])
def test_logits_far_from_zero(score, at):
    """Weights that are ratios of scores stay exact where the scores themselves vanish or saturate."""
    r = np.random.default_rng(11)
    M, E, k = 19, 48, 4
    l = (at + (abs(at) * 2.0 ** -12 + 1) * r.standard_normal((M, E))).astype(np.float32)
    lg = torch.from_numpy(l).cuda()
    check(lg, k, score, None, True, 1.0, None, r.standard_normal((M, k)).astype(np.float32), None, 1.0, f"{score} at {at}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_nan_and_infinite_logits(score, renorm, biased):
    M, E, k = 40, 70, 5
    lg = U.logits(M, E, F32, 4)
    lg[7, 30] = float("nan")
    lg[20, 69] = float("inf")
    clean = lg.clone()
    clean[7], clean[20] = 0.0, 0.0
    bias = torch.zeros(E).cuda() if biased else None
    how = dict(score=score, renormalise=renorm, bias=bias)
    ids, w, st = P.moe_router(lg.cuda(), k, stats=True, **how)
    cids, cw = P.moe_router(clean.cuda(), k, **how)
    rows = [t for t in range(M) if t not in (7, 20)]
    assert torch.equal(ids[rows], cids[rows]) and torch.equal(w[rows], cw[rows])
    assert bool(w[7].isnan().all()) and 30 not in ids[7].tolist() and len(set(ids[7].tolist())) == k
    assert int(ids[20, 0]) == 69 or (biased and score == "softmax")   # (there every score of the row is NaN)
    if score == "softmax":
        assert bool(w[20].isnan().all())
    else:
        assert bool(w[20].isfinite().all()) and float(w[20, 0]) >= float(w[20, 1])
    assert bool(st.balance.isnan().all()) and bool(st.means.isnan().all())
    g = P.moe_router_grad(lg.cuda(), ids, torch.ones_like(w), score=score, renormalise=renorm)
    assert bool(g[7].isnan().all()) and bool(g[rows].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_gradient_zeros_beside_a_gradient_that_is_not_finite(dtype, score, renorm, value):
    M, E, k = 30, 20, 3
    lg = U.logits(M, E, dtype, 12)
    lg[:, 4] = -float("inf")
    live = (torch.arange(M) % 3 - 1).to(torch.int32)
    how = dict(score=score, renormalise=renorm, live=live.cuda())
    ids, w, st = P.moe_router(lg.cuda(), k, stats=True, **how)
    dw = torch.full_like(w, value)
    for kw in (dict(d_weights=dw), dict(d_weights=dw, d_balance=torch.full((1,), value, device="cuda")),
               dict(d_weights=None, d_means=torch.full((E,), value, device="cuda"))):
        g = P.moe_router_grad(lg.cuda(), ids, stats=st, **kw, **how)
        assert not bool(g[live.cuda() < 0].ne(0.0).any()) and not bool(g[:, 4].ne(0.0).any())
        assert not bool(g[live.cuda() >= 0].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,k", [(8, 7), (64, 8), (64, 12), (256, 4)])
def test_a_nan_does_not_hide_the_rows_largest_logit(dtype, E, k):
    """Softmax with a bias: the row's weights are NaN, and its other experts are chosen as without it."""
    lg = U.logits(6, E, dtype, 14)
    lg[:, 2] = 200.0
    clean = lg.clone()
    clean[3, 1], lg[3, 1] = -float("inf"), float("nan")
    bias = torch.from_numpy(0.01 * np.random.default_rng(1).standard_normal(E).astype(np.float32)).cuda()
    ids, w = P.moe_router(lg.cuda(), k, bias=bias)
    want, cw = P.moe_router(clean.cuda(), k, bias=bias)
    assert torch.equal(ids, want) and bool(w[3].isnan().all()) and torch.equal(w[:3], cw[:3])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,k", [(24, 8), (24, 12), (129, 4), (700, 16)])
def test_an_infinite_logit_under_a_softmax_with_a_bias(dtype, E, k):
    """Its own score is NaN and never chosen, the others' are 0 (their biases decide), and the row's weights are NaN: the
    same for every top_k and wherever two biases are close or equal."""
    r = np.random.default_rng([E, k])
    lg = U.logits(6, E, dtype, 15)
    lg[1, 9], lg[4, 0], lg[4, 20] = float("inf"), float("inf"), float("inf")
    for bias in (r.standard_normal(E), np.zeros(E), 1.0 + r.permutation(E) * 2.0 ** -23):
        bias = bias.astype(np.float32)
        ids, w = P.moe_router(lg.cuda(), k, bias=torch.from_numpy(bias).cuda())
        for t in (1, 4):
            left = [e for e in range(E) if float(lg[t, e]) < float("inf")]
            want = sorted(left, key=lambda e: (-bias[e], e))[:k]
            assert ids[t].tolist() == want and bool(w[t].isnan().all())
        assert bool(w[[0, 2, 3, 5]].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E", [64, 129, 256])
def test_strided_and_unaligned_rows(dtype, E):
    r = np.random.default_rng(E)
    M, k = 45, 4
    lg = U.logits(M, E, dtype, 2)
    dw = torch.from_numpy(r.standard_normal((M, k)).astype(np.float32)).cuda()
    ids, w, st = P.moe_router(lg.cuda(), k, stats=True)
    one = torch.ones(1, device="cuda")
    g = P.moe_router_grad(lg.cuda(), ids, dw, stats=st, d_balance=one)
    for ld, off in ((E + 8, 0), (E + 3, 0), (E + 3, 1), (E, 1)):
        base = torch.full((M * ld + off,), float("nan")).to(dtype).cuda()
        view = base[off:].view(M, ld)[:, :E]
        view.copy_(lg)
        got = P.moe_router(view, k, stats=True)
        assert torch.equal(got[0], ids) and torch.equal(got[1], w)
        for a, b in zip(got[2], st):
            assert torch.equal(a, b)
        into = torch.full((M * ld + off,), 7.0).to(dtype).cuda()
        out = into[off:].view(M, ld)[:, :E]
        P.moe_router_grad(view, ids, dw, stats=st, d_balance=one, out=out)
        assert torch.equal(out, g)
        assert bool((into[:off] == 7.0).all()) and bool((into[off:].view(M, ld)[:, E:] == 7.0).all())
        P.moe_router_grad(view, ids, dw, stats=st, d_balance=one, out=view)       # over the logits
        assert torch.equal(view, g)


def test_many_tokens_and_repeatable_sums():
    M, E, k = 40013, 160, 6
    lg = U.logits(M, E, BF, 21).cuda()
    ids, w, st = P.moe_router(lg, k, score="sigmoid", renormalise=True, stats=True)
    l = lg.double()
    s = torch.sigmoid(l)
    q = s / s.sum(1, keepdim=True)
    order = torch.sort(lg.float(), dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(ids.long(), order)
    counts = torch.bincount(order.reshape(-1), minlength=E)
    assert torch.equal(st.counts.long(), counts) and int(st.tokens) == M
    err = U.router_error(np.array([12.0]), E) + (M // 4096 + 8) * ADD
    means = q.mean(0)
    assert_close(st.means, U.np64(means), err * U.np64(means), "means")
    loss = float(E * (counts.double() * means).sum() / counts.sum())
    assert abs(float(st.balance) - loss) <= err * loss
    work = torch.full((P.router_workspace(M, E),), 0xA5, dtype=torch.uint8, device="cuda")   # (its contents do not matter)
    again = P.moe_router(lg, k, score="sigmoid", renormalise=True, stats=True, work=work)
    for a, b in zip((*again[:2], *again[2]), (ids, w, *st)):
        assert torch.equal(a, b)


def test_ids_outside_the_experts_and_repeated_ids_in_the_gradient():
    """Device data is not trusted: entries outside [0, E) are skipped; an expert that stands twice gets both shares."""
    r = np.random.default_rng(2)
    M, E, k = 9, 24, 4
    lg = U.logits(M, E, F32, 5)
    ids = U.choose64(U.np64(lg), "softmax", None, k, None)
    dw = r.standard_normal((M, k)).astype(np.float32)
    bad, dropped = ids.copy(), ids.copy()
    bad[0, 1], bad[1, 2], bad[2, 0] = E, -7, 2 ** 30
    dropped[0, 1] = dropped[1, 2] = dropped[2, 0] = -1
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    assert torch.equal(P.moe_router_grad(lg.cuda(), dev(bad), dev(dw)), P.moe_router_grad(lg.cuda(), dev(dropped), dev(dw)))
    twice = ids.copy()
    twice[:, 1] = twice[:, 0]
    got = P.moe_router_grad(lg.cuda(), dev(twice), dev(dw))
    want, mag = U.router_grad64(U.np64(lg), "softmax", twice, False, 1.0, None, dw, None, None)
    assert_close(got, want, (2 * U.router_error(U.np64(lg), E) + 16 * ADD) * mag + 2 * U32 * np.abs(want), "twice")


def test_differentiable_form():
    r = np.random.default_rng(13)
    M, E, k = 50, 96, 4
    lg = U.logits(M, E, BF, 6).cuda().requires_grad_(True)
    bias = torch.from_numpy(0.1 * r.standard_normal(E).astype(np.float32)).cuda()
    rt = P.moe_experts_router(lg, k, score="sigmoid", bias=bias, renormalise=True, scale=2.0, means_grad=True)
    ids, w, st = P.moe_router(lg.detach(), k, score="sigmoid", bias=bias, renormalise=True, scale=2.0, stats=True)
    assert torch.equal(rt.ids, ids) and torch.equal(rt.weights, w) and torch.equal(rt.counts, st.counts)
    assert torch.equal(rt.means, st.means) and torch.equal(rt.balance, st.balance[0]) and rt.balance.dim() == 0
    assert not rt.ids.requires_grad and not rt.counts.requires_grad
    dw = torch.from_numpy(r.standard_normal((M, k)).astype(np.float32)).cuda()
    how = dict(score="sigmoid", renormalise=True, scale=2.0)
    one = lambda v: torch.full((1,), v, device="cuda")  # noqa: E731
    grads = lambda out, g=None: torch.autograd.grad(out, lg, g, retain_graph=True)[0]  # noqa: E731
    assert torch.equal(grads(rt.weights, dw), P.moe_router_grad(lg.detach(), ids, dw, **how))
    assert torch.equal(grads(rt.balance), P.moe_router_grad(lg.detach(), ids, None, stats=st, d_balance=one(1.0), **how))
    assert torch.equal(grads(rt.means.sum()), P.moe_router_grad(lg.detach(), ids, None, stats=st,
                                                                 d_means=torch.ones(E, device="cuda"), **how))
    assert torch.equal(grads((rt.weights * dw).sum() + 0.5 * rt.balance),
                       P.moe_router_grad(lg.detach(), ids, dw, stats=st, d_balance=one(0.5), **how))
    broadcast = grads(rt.weights.sum())           # a gradient that arrives with stride 0
    assert torch.equal(broadcast, P.moe_router_grad(lg.detach(), ids, torch.ones_like(w), **how))
    plain = P.moe_experts_router(lg, k, score="sigmoid", bias=bias, renormalise=True, scale=2.0)
    assert not plain.means.requires_grad and torch.equal(plain.means, rt.means) and torch.equal(plain.weights, rt.weights)
    assert torch.equal(torch.autograd.grad((plain.weights, plain.balance), lg, (dw, torch.full((), 0.5, device="cuda")))[0],
                       P.moe_router_grad(lg.detach(), ids, dw, stats=st, d_balance=one(0.5), **how))
    twice = torch.autograd.grad(P.moe_experts_router(lg, k).weights.pow(2).sum(), lg, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="once_differentiable"):
        twice.sum().backward()
    with pytest.raises(ValueError, match="top_k"):
        P.moe_experts_router(lg, E + 1)
    empty = P.moe_experts_router(torch.empty((0, E), dtype=BF, device="cuda", requires_grad=True), k)
    assert empty.ids.shape == (0, k) and float(empty.balance.detach()) == 0.0 and int(empty.counts.sum()) == 0
    empty.balance.backward()


def test_outputs_changed_in_place():
    """The loss, the weights and the means are tensors of their own: a program may scale or add to them in place."""
    lg = U.logits(20, 16, F32, 3).cuda().requires_grad_(True)
    for means_grad in (False, True):
        rt = P.moe_experts_router(lg, 4, means_grad=means_grad)
        grad = lambda t: torch.autograd.grad(t, lg, retain_graph=True)[0]  # noqa: E731
        want, value = grad(0.25 * rt.balance), float(rt.balance.detach())
        aux = rt.balance
        aux.mul_(0.25)
        aux += 1.0
        assert aux.dim() == 0 and abs(float(aux.detach()) - (0.25 * value + 1.0)) <= 4 * U32 * (value + 1.0)
        assert torch.equal(grad(aux), want)
        for t in (rt.weights, rt.means) if means_grad else (rt.weights,):
            want = grad((2.0 * t).sum())
            t.mul_(2.0)
            assert torch.equal(grad(t.sum()), want)


def test_replayed_graphs_and_two_streams():
    """A captured forward and gradient on changing logits, two graphs with a workspace each replayed side by side."""
    M, E, k = 200, 128, 4
    data = [U.logits(M, E, BF, s).cuda() for s in range(5)]
    dw = torch.ones((M, k), device="cuda")
    one = torch.ones(1, device="cuda")

    def step(lg, ids, w, st, work, out):
        P.moe_router(lg, k, renormalise=True, out=(ids, w), stats=st, work=work)
        P.moe_router_grad(lg, ids, dw, renormalise=True, stats=st, d_balance=one, out=out)

    def buffers():
        return (data[0].clone(), torch.empty((M, k), dtype=torch.int32, device="cuda"), torch.empty((M, k), device="cuda"),
                P.RouterStats(*(torch.empty(n, dtype=t, device="cuda") for n, t in
                                ((E, torch.int32), (E, F32), (1, F32), (1, torch.int32)))),
                torch.empty(P.router_workspace(M, E), dtype=torch.uint8, device="cuda"), torch.empty((M, E), dtype=BF, device="cuda"))

    sets, graphs, streams = [buffers(), buffers()], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for b in sets:
        step(*b)
    torch.cuda.synchronize()
    for b in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(*b)
        graphs.append(graph)
    for turn in range(4):
        for i, b in enumerate(sets):
            b[0].copy_(data[(turn + i) % 5])
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for i, b in enumerate(sets):
            want = buffers()
            want[0].copy_(data[(turn + i) % 5])
            step(*want)
            for got, ref in zip((*b[:3], *b[3], b[5]), (*want[:3], *want[3], want[5])):
                assert torch.equal(got, ref), (turn, i)


def test_captured_forward_and_backward_of_the_differentiable_form():
    M, E, k = 96, 64, 4
    data = [U.logits(M, E, F32, s).cuda() for s in range(4)]
    leaf = data[0].clone().requires_grad_(True)
    dw, share = torch.ones((M, k), device="cuda"), torch.full((), 0.1, device="cuda")
    how = dict(score="sigmoid", renormalise=True)

    def step(x):
        rt = P.moe_experts_router(x, k, **how)
        return rt.ids, rt.weights, rt.counts, rt.balance, torch.autograd.grad((rt.weights, rt.balance), x, (dw, share))[0]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                  # (a first pass outside, whose graph is gone before the capture)
        step(leaf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaf)
    for turn in range(4):
        with torch.no_grad():
            leaf.copy_(data[turn])
        graph.replay()
        torch.cuda.synchronize()
        want = step(data[turn].clone().requires_grad_(True))
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn
        del want


def test_refusals_of_the_wrappers():
    x = torch.zeros((4, 32), dtype=BF, device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for call, text in ((lambda: P.moe_router(x.half(), 2), "must be"), (lambda: P.moe_router(x[:, ::2], 2), "contiguous"),
                       (lambda: P.moe_router(x, 0), "top_k=0"), (lambda: P.moe_router(x, 33), "top_k=33"),
                       (lambda: P.moe_router(x, 2, bias=torch.zeros(31, device="cuda")), "bias"),
                       (lambda: P.moe_router(x, 2, live=ids[:, 0]), "live"),
                       (lambda: P.moe_router(x, 2, out=(ids[:3], torch.zeros((4, 2), device="cuda"))), "topk_ids"),
                       (lambda: P.moe_router(x, 2, stats=True, work=torch.zeros(8, dtype=torch.uint8, device="cuda")), "workspace"),
                       (lambda: P.moe_router_grad(x, ids[:3]), "topk_ids"),
                       (lambda: P.moe_router_grad(x, ids, d_balance=torch.ones(1, device="cuda")), "stats"),
                       (lambda: P.moe_router_grad(x, ids, torch.zeros((4, 3), device="cuda")), "d_weights")):
        with pytest.raises(ValueError, match=text):
            call()
