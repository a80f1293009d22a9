"""moe_fp8_quant and moe_act_fp8_quant against their definition: codes and scales bit for bit without
an activation (the arithmetic is fp32 throughout), within derived bounds with one."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests.experts_util import bf16

pytestmark = pytest.mark.gpu


def reference(v):
    """codes (bytes) and scales of fp32 v [R, K]."""
    R, K = v.shape
    G = -(-K // 128)
    codes, scales = np.zeros((R, K), np.uint8), np.zeros((R, G), np.float32)
    for g in range(G):
        part = v[:, g * 128: (g + 1) * 128]
        top = np.maximum(np.nanmax(np.abs(part), axis=1, initial=0.0), np.float32(2.0 ** -110)).astype(np.float32)
        scales[:, g] = top / np.float32(448)
        with np.errstate(invalid="ignore"):
            q = part * (np.float32(448) / top)[:, None]
        codes[:, g * 128: (g + 1) * 128] = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, scales


def same_codes(got, want):
    nan = (want & 0x7F) == 0x7F
    return np.array_equal(got[~nan], want[~nan]) and bool(((got[nan] & 0x7F) == 0x7F).all())


@pytest.mark.parametrize("R,K", [(1, 8), (1, 128), (3, 136), (5, 4096), (64, 2880), (257, 1000), (33, 7168)])
def test_codes_and_scales_are_exact(R, K):
    x = bf16((R, K), R * K)
    x[R // 2] *= 1000
    codes, scales = P.moe_fp8_quant(x.cuda())
    want_c, want_s = reference(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert same_codes(codes.view(torch.uint8).cpu().numpy(), want_c)


def test_zeros_infinities_nans_and_tiny_values():
    x = bf16((8, 384), 3)
    x[0] = 0
    x[1, :128] = 2.0 ** -120                      # below the floor of a group's maximum
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = float("nan")
    x[5, 200] = 3.3e38                            # bf16's largest
    x[6, 130] = -float("inf")
    x[7, 256:] = 2.0 ** -133                      # a subnormal
    codes, scales = P.moe_fp8_quant(x.cuda())
    want_c, want_s = reference(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert same_codes(codes.view(torch.uint8).cpu().numpy(), want_c)
    back = codes.float().cpu() * scales.cpu().repeat_interleave(128, 1)
    assert torch.isnan(back[2, :128]).all() and torch.isfinite(back[2, 128:]).all()
    assert torch.isnan(back[3, 7]) and torch.isfinite(back[3, :7]).all()


@pytest.mark.parametrize("kind,cols", [("none", 1), ("silu_mul", 2), ("swiglu_alpha", 2), ("relu2", 1)])
def test_dropped_rows_strides_and_activations(kind, cols):
    R, I = 37, 328
    h = bf16((R, cols * I), 11, 3.0)
    live = torch.from_numpy(np.random.default_rng(5).integers(-1, 3, R).astype(np.int32))
    live[0] = -1
    h[live < 0] = float("nan")
    base = torch.full((R, cols * I + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    base[:, : cols * I] = h.cuda()
    codes = torch.full((R, I + 16), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, 8), -1.0, device="cuda")
    out = (codes[:, :I], scales[:, :3])
    if kind == "none":
        P.moe_fp8_quant(base[:, :I], live.cuda(), out=out)
        v = h.double().numpy()
    else:
        P.moe_act_fp8_quant(kind, base[:, : cols * I], I, live.cuda(), alpha=1.5, limit=4.0, out=out)
        x = h.double().numpy()
        with np.errstate(over="ignore"):
            if kind == "silu_mul":
                v = x[:, :I] / (1 + np.exp(-x[:, :I])) * x[:, I:]
            elif kind == "relu2":
                v = np.maximum(x, 0) ** 2
            else:
                g, u = np.minimum(x[:, :I], 4.0), np.clip(x[:, I:], -4.0, 4.0)
                v = g / (1 + np.exp(-1.5 * g)) * (u + 1)
    on = live.numpy() >= 0
    assert (codes.cpu().numpy()[~on] == 0x55).all() and (scales.cpu().numpy()[~on] == -1.0).all()
    assert (codes.cpu().numpy()[:, I:] == 0x55).all() and (scales.cpu().numpy()[:, 3:] == -1.0).all()
    s = scales.cpu().numpy()[on, :3].astype(np.float64)
    c = codes.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)[on, :I]
    v = v[on]
    # the activation in fp32: an exponential of at most 30 (its argument rounded: 2^-24 * 30), a
    # reciprocal and three products: under 2^-18 relative
    rel = 2.0 ** -18
    for g in range(3):
        part, sc = v[:, g * 128: (g + 1) * 128], s[:, g]
        top = np.abs(part).max(axis=1)
        assert (np.abs(sc - top / 448) <= rel * top / 448).all()
        step = np.maximum(2.0 ** -4 * np.abs(part), 2.0 ** -10 * sc[:, None])     # half a step of e4m3
        assert (np.abs(c[:, g * 128: (g + 1) * 128] * sc[:, None] - part) <= step * (1 + rel) + 2 * rel * np.abs(part)).all()


def test_no_rows():
    codes, scales = P.moe_fp8_quant(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)


@pytest.mark.parametrize("kind,cols", [("silu_mul", 2), ("swiglu_alpha", 2), ("relu2", 1)])
@pytest.mark.parametrize("limit", [4.0, float("inf")])
def test_a_nan_before_the_activation_is_a_nan_code(kind, cols, limit):
    """Codes and scales of rows with NaNs are those with a gate of 0 (whose activation is 0) in their place,
    but for NaN codes there: a clamp or a maximum does not turn a NaN into a number."""
    R, I = 21, 328
    h = bf16((R, cols * I), 17, 3.0)
    at = torch.from_numpy(np.random.default_rng(18).random((R, I)) < 0.05)
    at[3, :128] = True                                    # a whole group
    at[4] = False
    clean = h.clone()
    clean[:, :I][at] = 0
    gate, up = h.clone(), h.clone()
    gate[:, :I][at] = float("nan")
    up[:, (cols - 1) * I:][at] = -float("nan")
    want_c, want_s = (t.cpu() for t in P.moe_act_fp8_quant(kind, clean.cuda(), I, alpha=1.5, limit=limit))
    for x in (gate, up):
        codes, scales = (t.cpu() for t in P.moe_act_fp8_quant(kind, x.cuda(), I, alpha=1.5, limit=limit))
        assert torch.equal(scales, want_s)
        assert torch.equal(torch.isnan(codes.float()), at)
        assert torch.equal(codes.view(torch.uint8)[~at], want_c.view(torch.uint8)[~at])
