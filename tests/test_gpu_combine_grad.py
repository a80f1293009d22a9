"""Gradients of the weighted combine, without and with the post-expert norm, against their plain 64-bit form."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests import ends_util as U
from tests.experts_util import U16, U32, assert_close, bf16, strided
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
EPS = 1e-5


def inputs(M, k, H, seed, dead=0.2):
    r = np.random.default_rng([seed, 82])
    y, dout = bf16((M * k, H), seed), bf16((M, H), seed + 1)
    g = torch.from_numpy(r.standard_normal((M, k)).astype(np.float32))
    local = torch.from_numpy(np.where(r.random((M, k)) < dead, -1, r.integers(0, 9, (M, k))).astype(np.int32))
    norm = (1.0 + 0.3 * torch.from_numpy(r.standard_normal(H).astype(np.float32))).bfloat16()
    return y, g, local, dout, norm


def check(y, g, local, dout, norm, c, got, what):
    (M, k), H = g.shape, y.shape[1]
    _, dy, dg, dn, dy_b, dg_b, dn_b = U.combine64(U.np64(y).reshape(M, k, H), U.np64(g), local.cpu().numpy() >= 0,
                                                   None if norm is None else U.np64(norm), EPS, c, U.np64(dout))
    tiny = 2.0 ** -125
    assert_close(got[0], dy, dy_b * (1 + U16) + U16 * np.abs(dy) + tiny, what + " dy")
    assert_close(got[1], dg, dg_b * (1 + U32) + U32 * np.abs(dg) + tiny, what + " dg")
    if norm is not None:
        assert_close(got[2], dn, dn_b * (1 + U16) + U16 * np.abs(dn) + tiny, what + " dn")


SIZES = [(1, 1, 8), (3, 2, 16), (70, 2, 512), (5, 3, 520), (33, 4, 2880), (9, 8, 4096), (6, 8, 4104), (4, 8, 8192), (3, 8, 8200),
         (2, 5, 12288), (7, 9, 264), (5, 16, 4096), (700, 2, 72), (1100, 1, 136)]


@pytest.mark.parametrize("M,k,H", SIZES)
@pytest.mark.parametrize("norm", [False, True])
def test_gradients(M, k, H, norm):
    y, g, local, dout, n = inputs(M, k, H, M + k + H)
    n = n if norm else None
    yd = y.cuda()
    yd[(local < 0).view(-1).cuda()] = float("nan")                  # rows of dead slots are not read
    announce(f"M={M} k={k} H={H} norm={norm}")
    args = (yd, g.cuda(), local.cuda(), dout.cuda())
    how = dict(norm_w=None if n is None else n.cuda(), eps=EPS, routed_scaling_factor=1.5)
    got = P.moe_combine_grad(*args, **how)
    check(y, g, local, dout, n, 1.5, got, f"M={M} k={k} H={H}")
    again = P.moe_combine_grad(*args, **how)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
    for keep in ((0,), (1,), (2,), (0, 2), (1, 2), (0, 1)):         # some of the gradients alone
        if not norm and 2 in keep:
            continue
        out = [torch.full_like(t, 3.0) if i in keep else None for i, t in enumerate(got)]
        P.moe_combine_grad(*args, out=out, **how)
        assert all(t is None or torch.equal(t, got[i]) for i, t in enumerate(out)), keep


def test_norm_weights_of_more_columns_than_a_gradient_takes():
    y, g, local, dout, n = inputs(2, 2, 16384, 5)
    args, how = (y.cuda(), g.cuda(), local.cuda(), dout.cuda()), dict(norm_w=n.cuda(), eps=EPS)
    with pytest.raises(ValueError, match="d_norm_w of 16384 columns"):
        P.moe_combine_grad(*args, **how)
    out = (torch.empty_like(args[0]), torch.empty_like(args[1]), None)
    got = P.moe_combine_grad(*args, out=out, **how)
    _, dy, dg, _, dy_b, dg_b, _ = U.combine64(U.np64(y).reshape(2, 2, -1), U.np64(g), local.numpy() >= 0, U.np64(n), EPS, 1.0,
                                              U.np64(dout))
    assert_close(got[0], dy, dy_b * (1 + U16) + U16 * np.abs(dy), "dy")
    assert_close(got[1], dg, dg_b * (1 + U32) + U32 * np.abs(dg), "dg")


@pytest.mark.parametrize("norm", [False, True])
def test_all_slots_dead_and_zero_rows(norm):
    M, k, H = 20, 3, 256
    y, g, local, dout, n = inputs(M, k, H, 3)
    how = dict(norm_w=n.cuda() if norm else None, eps=EPS)
    none = torch.full_like(local, -1)
    for t in P.moe_combine_grad(torch.full_like(y, float("nan")).cuda(), g.cuda(), none.cuda(), dout.cuda(), **how):
        assert t is None or float(t.abs().max()) == 0.0
    y[::2] = 0.0                                                    # a row of zeros: the norm is eps's
    check(y, g, local, dout, n if norm else None, 1.0, P.moe_combine_grad(y.cuda(), g.cuda(), local.cuda(), dout.cuda(), **how), "zeros")


@pytest.mark.parametrize("norm", [False, True])
def test_differentiable_form(norm):
    M, k, H = 37, 4, 320
    y, g, local, dout, n = inputs(M, k, H, 8)
    leaves = [t.cuda().requires_grad_(True) for t in ((y, g, n) if norm else (y, g))]
    nw = leaves[2] if norm else None
    out = P.moe_experts_combine(leaves[0], leaves[1], local.cuda(), norm_w=nw, eps=EPS, routed_scaling_factor=0.7)
    ref = P.moe_combine(y.cuda(), g.cuda(), local.cuda(), norm_w=n.cuda() if norm else None, eps=EPS, routed_scaling_factor=0.7)
    assert torch.equal(out, ref)
    how = dict(norm_w=n.cuda() if norm else None, eps=EPS, routed_scaling_factor=0.7)
    plain = lambda d: P.moe_combine_grad(y.cuda(), g.cuda(), local.cuda(), d, **how)  # noqa: E731
    forms = [dout.cuda(), strided(dout, H + 8), strided(dout, H + 3),
             torch.cat([torch.zeros(1, dtype=torch.bfloat16), dout.reshape(-1)]).cuda()[1:].view(M, H),       # 2-byte aligned
             dout.cuda().t().contiguous().t(), torch.ones((), dtype=torch.bfloat16, device="cuda").expand(M, H)]
    for d in forms:
        got = torch.autograd.grad(out, leaves, d, retain_graph=True)
        for a, b in zip(got, plain(d.clone(memory_format=torch.contiguous_format))):
            assert torch.equal(a, b)
    for i, leaf in enumerate(leaves):                               # one leaf at a time
        fixed = [t.detach().requires_grad_(j == i) for j, t in enumerate(leaves)]
        o = P.moe_experts_combine(fixed[0], fixed[1], local.cuda(), norm_w=fixed[2] if norm else None, eps=EPS, routed_scaling_factor=0.7)
        assert torch.equal(torch.autograd.grad(o, fixed[i], dout.cuda())[0], plain(dout.cuda())[i])
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    gw = torch.empty((0, k), device="cuda", requires_grad=True)
    o = P.moe_experts_combine(e, gw, torch.empty((0, k), dtype=torch.int32, device="cuda"), norm_w=nw)
    o.sum().backward()
    assert e.grad.shape == (0, H) and gw.grad.shape == (0, k)
    assert not norm or float(leaves[2].grad.abs().max()) == 0.0     # no tokens, no share


def test_a_step_whose_gradient_would_be_refused_is_refused_at_once():
    y, g, local, _, n = (t.cuda() for t in inputs(2, 2, 16384, 5))
    n.requires_grad_(True)
    with pytest.raises(ValueError, match="12288"):
        P.moe_experts_combine(y, g, local, norm_w=n)
    with torch.no_grad():
        assert P.moe_experts_combine(y, g, local, norm_w=n).shape == (2, 16384)
    y.requires_grad_(True)                                          # the others' gradients have no such limit
    P.moe_experts_combine(y, g, local, norm_w=n.detach()).sum().backward()
    M = 1 << 24
    y, g = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda"), torch.zeros((M, 1), device="cuda")
    local = torch.zeros((M, 1), dtype=torch.int32, device="cuda")
    assert P.moe_experts_combine(y, g, local).shape == (M, 8)
    with pytest.raises(ValueError, match="2\\^24"):
        P.moe_experts_combine(y.requires_grad_(True), g, local)


def test_offsets_past_four_gigabytes():
    """y of 4.3 GB: the last token's gradients are those of a batch of its own."""
    M, k, H = 65600, 8, 4096
    y = torch.zeros((M * k, H), dtype=torch.bfloat16, device="cuda")
    small = inputs(4, k, H, 31, dead=0.0)
    y[-4 * k:] = small[0].cuda()
    g, local = torch.ones((M, k), device="cuda"), torch.full((M, k), -1, dtype=torch.int32, device="cuda")
    g[-4:], local[-4:] = small[1].cuda(), small[2].cuda()
    dout = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    dout[-4:] = small[3].cuda()
    for n in (None, small[4].cuda()):
        got = P.moe_combine_grad(y, g, local, dout, norm_w=n, eps=EPS)
        own = P.moe_combine_grad(small[0].cuda(), small[1].cuda(), small[2].cuda(), small[3].cuda(), norm_w=n, eps=EPS)
        assert torch.equal(got[0][-4 * k:], own[0]) and torch.equal(got[1][-4:], own[1])
        assert not bool(got[0][: -4 * k].any()) and not bool(got[1][:-4].any())
        if n is not None:
            assert_close(got[2], U.np64(own[2]), 4 * U16 * np.abs(U.np64(own[2])) + 1e-6 * float(own[2].abs().max()), "dn")


def test_replayed_graph():
    M, k, H = 600, 4, 384
    sets = [inputs(M, k, H, s) for s in (1, 2, 3)]
    y, g, local, dout, n = (t.cuda() for t in sets[0])
    out = [torch.empty_like(y), torch.empty_like(g), torch.empty_like(n)]
    work = torch.empty(P.combine_grad_workspace(M, H), device="cuda")
    call = lambda o, w: P.moe_combine_grad(y, g, local, dout, norm_w=n, eps=EPS, out=o, work=w)  # noqa: E731
    call(out, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, work)
    for turn in range(4):
        for t, s in zip((y, g, local, dout, n), sets[turn % 3]):
            t.copy_(s)
        work.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = call([torch.empty_like(t) for t in out], None)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), turn


def test_captured_forward_and_backward_of_the_differentiable_form():
    M, k, H = 40, 2, 256
    sets = [inputs(M, k, H, s, dead=0.0) for s in (1, 2, 3)]
    local = sets[0][2].cuda()
    leaves = [sets[0][i].cuda().requires_grad_(True) for i in (0, 1, 4)]
    dout = sets[0][3].cuda()

    def step(a):
        o = P.moe_experts_combine(a[0], a[1], local, norm_w=a[2], eps=EPS)
        return (o, *torch.autograd.grad(o, a, dout))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(leaves)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaves)
    for turn in range(4):
        s = sets[turn % 3]
        with torch.no_grad():
            for leaf, i in zip(leaves, (0, 1, 4)):
                leaf.copy_(s[i])
        graph.replay()
        torch.cuda.synchronize()
        want = step([s[i].cuda().requires_grad_(True) for i in (0, 1, 4)])
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn
        del want


def test_more_tokens_than_workgroups():
    M, H = (1 << 20) + 777, 8
    y, g, local, dout, _ = inputs(M, 1, H, 77, dead=0.1)
    got = P.moe_combine_grad(y.cuda(), g.cuda(), local.cuda(), dout.cuda())
    check(y, g, local, dout, None, 1.0, got, "many")


def test_refusals_of_the_wrappers():
    y, g, local, dout, n = (t.cuda() for t in inputs(4, 2, 64, 1))
    for call, text in ((lambda: P.moe_combine_grad(y[:7], g, local, dout), "must have a row"),
                       (lambda: P.moe_combine_grad(y, g, local[:3], dout), "slot_local_ids"),
                       (lambda: P.moe_combine_grad(y, g, local, dout[:3]), "d_out"),
                       (lambda: P.moe_combine_grad(y, g, local, dout, norm_w=n[:32].contiguous()), "norm_w"),
                       (lambda: P.moe_combine_grad(y, g, local, dout, out=(None, None, n)), "norm_w"),
                       (lambda: P.moe_combine_grad(y, g, local, dout, norm_w=n, work=torch.zeros(8, device="cuda")), "workspace"),
                       (lambda: P.moe_experts_combine(y.float(), g, local), "must be"),
                       (lambda: P.moe_experts_combine(y, g.double(), local), "topk_weights")):
        with pytest.raises(ValueError, match=text):
            call()
