"""A training step of the whole expert layer from the router's logits to its output and back -- router, align,
experts' products, combine, balance loss -- and a serving step with adapters beside the shared projection."""
import dataclasses

import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
import workloads
from tests import ends_util as U
from tests.experts_util import aligned
from tests.gpu_util import layer_violations, make_layer, oracle_layer

pytestmark = pytest.mark.gpu


def silu_mul(h):
    gate, up = h.float().chunk(2, dim=-1)
    return (gate * torch.sigmoid(gate) * up).bfloat16()


@pytest.mark.parametrize("score,norm,start,E_local", [("softmax", False, 0, 8), ("sigmoid", True, 2, 4)])
def test_training_step_from_logits_to_output(score, norm, start, E_local):
    """Against the same layer in fp32 torch operations on the same choices.  The bf16 steps between (each off by
    2^-8, about ten of them in a row, errors of either sign) leave 2 % of a gradient's size."""
    torch.manual_seed(3)
    M, D, I, E, k, B = 200, 64, 128, 8, 2, 16
    mk = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    x, wr = mk(M, D).bfloat16(), (mk(E, D) / 8).bfloat16()
    w13, w2 = (mk(E_local, 2 * I, D) / 8).bfloat16(), (mk(E_local, D, I) / 11).bfloat16()
    nw = (1 + 0.1 * mk(D)).bfloat16() if norm else None
    live = torch.where(torch.arange(M, device="cuda") % 25 > 21, -1, 0).to(torch.int32)
    target = mk(M, D)
    leaves = [t.detach().clone().requires_grad_(True) for t in (x, wr, w13, w2) + ((nw,) if norm else ())]

    def loss_of(out, balance):
        return (out.float() * target).sum() / M + 0.3 * balance

    a = leaves
    rt = P.moe_experts_router(a[0] @ a[1].t(), k, score=score, renormalise=True, scale=1.5, live=live)
    al = P.moe_align(rt.ids, start, E_local, B)
    h = P.moe_experts_linear(a[0], a[2], al, k, B)
    y = P.moe_experts_linear(silu_mul(h), a[3], al, 1, B)
    out = P.moe_experts_combine(y, rt.weights, al[3], norm_w=a[4] if norm else None, eps=1e-6)
    got = torch.autograd.grad(loss_of(out, rt.balance), a)

    b = [t.detach().float().requires_grad_(True) for t in leaves]
    on = (live >= 0).float()[:, None]
    logits = (a[0] @ a[1].t()).detach().float() + ((b[0] @ b[1].t()) - (b[0] @ b[1].t()).detach())   # the same values
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    q = s / s.sum(1, keepdim=True)
    at = rt.ids.clamp_min(0).long()
    w = torch.gather(s, 1, at) * on
    w = 1.5 * w / w.sum(1, keepdim=True).clamp_min(1e-30)
    local = torch.where((rt.ids >= start) & (rt.ids < start + E_local), rt.ids - start, -1)
    ref = torch.zeros((M, D), device="cuda")
    for e in range(E_local):
        for c in range(k):
            mask = (local[:, c] == e).float()[:, None]
            gate, up = (b[0] @ b[2][e].t()).chunk(2, dim=1)
            z = (gate * torch.sigmoid(gate) * up) @ b[3][e].t()
            if norm:
                z = z * b[4]
                z = z / torch.sqrt((z * z).mean(1, keepdim=True) + 1e-6)
            ref = ref + mask * w[:, c: c + 1] * z
    counts = torch.bincount(rt.ids[rt.ids >= 0].long(), minlength=E).float()
    assert torch.equal(counts.int(), rt.counts)
    balance = E * (counts / counts.sum() * (q * on).sum(0) / on.sum()).sum()
    assert abs(float(balance.detach()) - float(rt.balance.detach())) < 1e-5 * float(balance.detach())
    want = torch.autograd.grad(loss_of(ref, balance), b)
    rms = lambda t: float(t.double().pow(2).mean().sqrt())  # noqa: E731
    assert rms(out.float() - ref) < 0.01 * rms(ref)
    for i, (g, r) in enumerate(zip(got, want)):
        assert rms(g.float() - r) < 0.02 * rms(r), (i, rms(g.float() - r), rms(r))
    assert float(out[live < 0].abs().max()) == 0.0


def test_serving_step_with_adapters_beside_the_shared_projection():
    """moe_fp8_quant -> moe_w8a8_linear -> moe_adapters_add in place: the sum of the projection's rows and of the
    adapters' own, and one align for two projections."""
    torch.manual_seed(4)
    M, K, N, n, r, B = 70, 256, 384, 5, 16, 16
    x = torch.randn((M, K), device="cuda").bfloat16()
    W = (torch.randn((N, K), device="cuda") * 50).to(torch.float8_e4m3fn)
    ws = torch.full((N // 128, K // 128), 1e-3, device="cuda")
    ids = np.random.default_rng(1).integers(-1, n, (M, 1)).astype(np.int32)
    plan, _ = aligned(ids, 0, n, B)
    q, qs = P.moe_fp8_quant(x)
    base = P.moe_w8a8_linear(q, qs, W, ws)
    for seed in (1, 2):
        A = (torch.randn((n, r, K), device="cuda") / 16).bfloat16()
        Bm = (torch.randn((n, N, r), device="cuda") / 4).bfloat16()
        y = base.clone()
        P.moe_adapters_add(y, x, A, Bm, plan, B, out=y)
        want, bound = U.adapters64(U.np64(base), U.np64(x), U.np64(A), U.np64(Bm), None, None, ids.reshape(-1), 1)
        assert (np.abs(U.np64(y) - want) <= bound * 1.01 + 2.0 ** -8 * np.abs(want)).all()


def test_routed_layer_takes_the_routers_output():
    """The W4A16 layer on the router's ids and weights: padding tokens come out as zeros, the others as the oracle's."""
    wl = workloads.small_workload("nvfp4_g16")
    lw, inp = workloads.make_weights(wl), workloads.make_inputs(wl, 45)
    x, ids, _ = workloads.device_inputs(inp)
    logits = torch.randn((45, wl.n_global), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    live = torch.where(torch.arange(45, device="cuda") % 9 == 8, -1, 0).to(torch.int32)
    ids, weights = P.moe_router(logits, wl.top_k, score="sigmoid", renormalise=True, live=live)
    got = workloads.bf16_to_float(make_layer(wl, lw)(x, ids, weights))
    routed = dataclasses.replace(inp, topk_ids=ids.cpu().numpy(), topk_weights=weights.cpu().numpy())
    assert layer_violations(got, oracle_layer(wl, lw, routed)) == 0
    assert not got[8::9].any() and got[:8].any()
