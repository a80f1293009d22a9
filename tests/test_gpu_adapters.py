"""Low-rank adapters of many requests beside a shared projection against their plain 64-bit form."""
import numpy as np
import pytest
import torch

import quantized_mixture_experts_align_amd as P
from tests import ends_util as U
from tests.experts_util import U16, aligned, assert_close, bf16, strided
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


def make(numel, n, r, N, K, seed, top_k=1, none=0.2):
    rng = np.random.default_rng([seed, 83])
    ids = np.where(rng.random(numel) < none, -1, rng.integers(0, n, numel)).astype(np.int32)
    return dict(base=bf16((numel, N), seed), x=bf16((numel // top_k, K), seed + 1), A=bf16((n, r, K), seed + 2, K ** -0.5),
                B=bf16((n, N, r), seed + 3, r ** -0.5), scales=torch.from_numpy(rng.uniform(0.2, 2.0, n).astype(np.float32)),
                ranks=None, ids=ids, top_k=top_k)


def reference(d):
    return U.adapters64(U.np64(d["base"]), U.np64(d["x"]), U.np64(d["A"]), U.np64(d["B"]),
                        None if d["scales"] is None else U.np64(d["scales"]), None if d["ranks"] is None else d["ranks"].numpy(),
                        d["ids"], d["top_k"])


def call(d, B, base=None, x=None, **more):
    n = d["A"].shape[0]
    al, _ = aligned(d["ids"].reshape(-1, 1), 0, n, B)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    return P.moe_adapters_add(d["base"].cuda() if base is None else base, d["x"].cuda() if x is None else x, c(d["A"]), c(d["B"]),
                              al, B, scales=c(d["scales"]), ranks=c(d["ranks"]), top_k=d["top_k"], **more)


def check(d, got, what):
    want, bound = reference(d)
    assert_close(got, want, bound * (1 + U16) + U16 * np.abs(want), what)


SIZES = [(1, 1, 8, 8, 8, 16), (1, 8, 16, 4096, 7168, 16), (3, 4, 24, 72, 40, 1), (64, 64, 16, 1032, 1032, 16), (50, 3, 32, 264, 4104, 5),
         (40, 5, 40, 520, 136, 17), (100, 4, 64, 256, 512, 32), (300, 3, 64, 1000, 264, 64), (257, 2, 72, 88, 328, 100),
         (500, 6, 128, 136, 96, 256), (90, 3, 200, 328, 200, 16), (140, 2, 256, 264, 520, 64), (2000, 7, 16, 136, 72, 64),
         (700, 512, 8, 64, 64, 16), (20, 1, 16, 24, 24, 48), (9, 3, 32, 520, 2056, 16), (30, 12, 16, 1032, 4104, 8),
         (16, 1, 16, 8200, 8184, 16), (300, 40, 24, 600, 504, 16), (600, 40, 32, 88, 520, 16),
         (9, 3, 32, 520, 2040, 16), (5, 1, 32, 264, 4088, 16), (30, 12, 16, 1032, 4096, 8)]


@pytest.mark.parametrize("numel,n,r,N,K,B", SIZES)
@pytest.mark.parametrize("scaled", [True, False])
def test_rows_of_many_adapters(numel, n, r, N, K, B, scaled):
    d = make(numel, n, r, N, K, numel + n + r)
    if not scaled:
        d["scales"] = None
    what = f"numel={numel} n={n} r={r} N={N} K={K} B={B}"
    announce(what)
    got = call(d, B)
    check(d, got, what)
    assert torch.equal(call(d, B), got)
    plain = torch.from_numpy(d["ids"] < 0).cuda()
    assert torch.equal(got[plain], d["base"].cuda()[plain])
    y = d["base"].cuda()
    assert call(d, B, base=y, out=y) is y and torch.equal(y, got)                                        # in place


@pytest.mark.parametrize("B", [16, 64])
def test_ranks_of_their_own(B):
    """What stands behind an adapter's rank -- here NaN -- is not used; ranks outside 0..r are clamped."""
    numel, n, r, N, K = 130, 8, 72, 200, 168
    d = make(numel, n, r, N, K, 7, none=0.1)
    d["ranks"] = torch.tensor([0, 1, 7, 8, 33, 72, -5, 1000], dtype=torch.int32)
    for a, own in enumerate(d["ranks"].clamp(0, r).tolist()):
        d["A"][a, own:], d["B"][a, :, own:] = float("nan"), float("nan")
    clean = {**d, "A": d["A"].nan_to_num(0.0), "B": d["B"].nan_to_num(0.0)}
    got = call(d, B)
    check(clean, got, "ranks")
    none = torch.from_numpy(np.isin(d["ids"], (0, 6))).cuda()
    assert torch.equal(got[none], d["base"].cuda()[none])                                                # adapters of rank 0


@pytest.mark.parametrize("top_k,B", [(2, 16), (4, 64)])
def test_slots_of_several_choices_share_a_row(top_k, B):
    d = make(240, 6, 16, 136, 264, 9, top_k=top_k)
    check(d, call(d, B), f"top_k={top_k}")


def test_strided_rows_and_padding_columns():
    d = make(77, 4, 16, 200, 120, 10)
    base, x = strided(d["base"], 232), strided(d["x"], 136)
    into = torch.full((77, 240), 5.0, dtype=torch.bfloat16, device="cuda")
    got = call(d, 16, base=base, x=x, out=into[:, :200])
    check(d, got, "strided")
    assert bool((into[:, 200:] == 5.0).all())
    inner = strided(d["base"], 232)
    call(d, 16, base=inner, x=x, out=inner)
    assert torch.equal(inner, got)


@pytest.mark.parametrize("numel,n,r,N,B", [(1, 1, 16, 4096, 16), (16, 8, 16, 1032, 16), (40, 3, 32, 512, 16), (70, 5, 24, 1544, 16),
                                           (9, 3, 32, 4096, 16), (64, 64, 16, 8192, 16), (100, 4, 64, 776, 64)])
def test_out_over_x(numel, n, r, N, B):
    """x += B A x in place, and out over x with base elsewhere: all of x is read before a column is written."""
    d = make(numel, n, r, N, N, 3 * numel + r)
    announce(f"over x: numel={numel} n={n} r={r} N=K={N} B={B}")
    h = d["x"].cuda()
    assert call(d, B, base=h, x=h, out=h) is h
    check({**d, "base": d["x"]}, h, "base = x = out")
    h = d["x"].cuda()
    call(d, B, x=h, out=h)
    check(d, h, "x = out")
    both = torch.empty((numel + 3, N), dtype=torch.bfloat16, device="cuda")
    x = both[3:].copy_(d["x"])
    check(d, call(d, B, x=x, out=both[:-3]), "out ends in x")


def test_out_over_x_of_several_choices():
    d = make(48, 5, 16, 1032, 1032, 23, top_k=2)
    out = torch.empty((48, 1032), dtype=torch.bfloat16, device="cuda")
    x = out[20:44].copy_(d["x"])
    check(d, call(d, 16, x=x, out=out), "out around x")


def test_out_in_other_columns_of_bases_rows():
    """base, out and x as columns of one buffer's rows: they share no element."""
    d = make(40, 4, 16, 200, 200, 26)
    buf = torch.full((40, 640), 9.0, dtype=torch.bfloat16, device="cuda")
    base, out, x = buf[:, 208:408], buf[:, :200], buf[:, 416:616]
    base.copy_(d["base"]), x.copy_(d["x"])
    for o in (out, buf[:, 8:208]):
        check(d, call(d, 16, base=base, x=x, out=o), "columns")
    assert torch.equal(base.cpu(), d["base"]) and torch.equal(x.cpu(), d["x"])
    assert bool((buf[:, 616:] == 9.0).all()) and bool((buf[:, 408:416] == 9.0).all())
    for o in (buf[:, 16:216], buf[:, 400:600]):
        with pytest.raises(ValueError, match="overlaps base"):
            call(d, 16, base=base, x=x, out=o)


def test_no_row_all_rows_and_one_row_of_an_adapter():
    for none in (1.0, 0.0):
        d = make(33, 3, 8, 64, 64, 12, none=none)
        check(d, call(d, 16), f"none={none}")
    d = make(90, 4, 16, 72, 72, 13)
    d["ids"][:] = 2
    d["ids"][41] = 0                                  # an adapter of one row, one of 89, two of none
    check(d, call(d, 64), "uneven")
    d = make(0, 3, 8, 64, 64, 14)
    assert call(d, 16).shape == (0, 64)


def test_large_values_and_infinities():
    d = make(24, 2, 8, 64, 64, 15, none=0.0)
    d["x"] = (d["x"].float() * 2.0 ** 60).bfloat16()
    d["A"] = (d["A"].float() * 2.0 ** 30).bfloat16()
    check(d, call(d, 16), "large")
    d = make(24, 2, 8, 64, 64, 16, none=0.0)
    d["x"][5, 9] = float("inf")                       # its own row alone
    d["x"][6, 3] = float("nan")
    got = call(d, 16)
    rows = [m for m in range(24) if m not in (5, 6)]
    want, bound = reference({**d, "x": d["x"].nan_to_num(0.0, 0.0)})
    assert_close(got[rows], want[rows], (bound * (1 + U16) + U16 * np.abs(want))[rows], "others")
    assert not bool(got[5].isfinite().any()) and bool(got[6].isnan().all())


def test_stale_entries_behind_the_live_blocks_are_not_used():
    d = make(60, 5, 16, 136, 136, 17)
    al, _ = aligned(d["ids"].reshape(-1, 1), 0, 5, 16)
    end = int(al[2])
    al[0][end:] = 3                                   # entries of an earlier, longer batch
    al[1][end // 16:] = 1
    got = P.moe_adapters_add(d["base"].cuda(), d["x"].cuda(), d["A"].cuda(), d["B"].cuda(), al, 16, scales=d["scales"].cuda())
    check(d, got, "stale")


def test_offsets_past_four_gigabytes():
    """Rows far apart: base, out and x in buffers of 6 GB, B of more than 2^31 values."""
    numel, ld = 48, 1 << 26
    d = make(numel, 3, 16, 128, 256, 18)
    far = lambda t: torch.as_strided(torch.empty((numel - 1) * ld + t.shape[1], dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                                     t.shape, (ld, 1)).copy_(t.cuda())
    out = far(torch.zeros((numel, 128)))
    check(d, call(d, 16, base=far(d["base"]), x=far(d["x"]), out=out), "far rows")
    torch.cuda.empty_cache()
    n, N, r = 300, 32768, 256                         # B: 2.5e9 values; only the last adapters are used
    A, B = torch.zeros((n, r, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, N, r), dtype=torch.bfloat16, device="cuda")
    small = make(20, 2, r, N, 64, 19, none=0.0)
    A[-2:], B[-2:] = small["A"].cuda(), small["B"].cuda()
    al, _ = aligned((small["ids"] + n - 2).reshape(-1, 1).astype(np.int32), 0, n, 16)
    small["scales"] = None
    check(small, P.moe_adapters_add(small["base"].cuda(), small["x"].cuda(), A, B, al, 16), "far adapters")


def test_replayed_graphs_with_workspaces_of_their_own():
    numel, n, r, N, K, B = 96, 6, 16, 264, 520, 16
    d = make(numel, n, r, N, K, 20)
    base, x, A, Bm, s = (d[key].cuda() for key in ("base", "x", "A", "B", "scales"))
    batches = [aligned(np.random.default_rng(t).integers(-1, n, (numel, 1)).astype(np.int32), 0, n, B)[0] for t in range(4)]
    sets = []
    for i in range(2):
        al = tuple(t.clone() for t in batches[i])
        out = torch.empty_like(base)
        work = torch.empty(P.adapters_workspace(numel, n, r, K, B), device="cuda")
        run = lambda al=al, out=out, work=work: P.moe_adapters_add(base, x, A, Bm, al, B, scales=s, out=out, work=work)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        sets.append((graph, al, out, torch.cuda.Stream()))
    for turn in range(4):
        for i, (_, al, _, _) in enumerate(sets):
            for t, v in zip(al, batches[(turn + i) % 4]):
                t.copy_(v)
        torch.cuda.synchronize()
        for graph, _, _, stream in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for i, (_, _, out, _) in enumerate(sets):
            assert torch.equal(out, P.moe_adapters_add(base, x, A, Bm, batches[(turn + i) % 4], B, scales=s)), (turn, i)


def test_a_base_that_autograd_holds_is_known_to_have_changed():
    d = make(20, 3, 16, 64, 64, 24)
    w = torch.ones((20, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    for into, mode in ((None, torch.enable_grad), (None, torch.no_grad), (torch.zeros_like(w).detach(), torch.enable_grad)):
        y = d["base"].cuda()
        z = w * (y if into is None else into)                       # (keeps it for w's gradient)
        with mode():
            call(d, 16, base=y, out=y if into is None else into)
        with pytest.raises(RuntimeError, match="inplace operation"):
            z.sum().backward()
    want = call(d, 16)
    with torch.inference_mode():
        y = d["base"].cuda()
        assert torch.equal(call(d, 16, base=y, out=y), want)
        y = d["base"].cuda()
    assert torch.equal(call(d, 16, base=y, out=y), want)            # a tensor of inference mode, outside of it


def test_refusals_of_the_wrapper():
    d = make(12, 2, 8, 64, 64, 21)
    al, _ = aligned(d["ids"].reshape(-1, 1), 0, 2, 16)
    base, x, A, B = (d[key].cuda() for key in ("base", "x", "A", "B"))
    ok = dict(base=base, x=x, A=A, B=B, align=al, block_m=16)
    for change, text in ((dict(x=x[:11]), "rows"), (dict(A=A[:, :, :32]), "columns of x"), (dict(B=B[:, :32]), "B must be"),
                         (dict(A=A.float()), "must be"), (dict(out=base[1:]), "out must be"), (dict(out=x.view(12, 64)[:, :32]), "out"),
                         (dict(scales=torch.ones(3, device="cuda")), "scales"), (dict(ranks=torch.ones(2, device="cuda")), "ranks"),
                         (dict(block_m=1), "align's outputs"), (dict(work=torch.ones(4, device="cuda")), "workspace"),
                         (dict(align=(*al[:3], al[3][:3])), "slot_local_ids"), (dict(top_k=2), "rows")):
        with pytest.raises(ValueError, match=text):
            P.moe_adapters_add(**{**ok, **change})


# r, K: on both sides of the sizes at which few rows take one launch instead of two, in each width of the staged columns
@pytest.mark.parametrize("r", [16, 24, 32, 64, 72])
@pytest.mark.parametrize("numel,K,B", [(1, 264, 16), (1, 8200, 16), (40, 264, 16), (40, 4104, 16), (40, 264, 64), (300, 1032, 32)])
def test_ranks_of_their_own_in_both_forms(r, numel, K, B):
    """What stands behind an adapter's own rank -- here NaN -- is not used."""
    n = 5
    d = make(numel, n, r, 520, K, 7 * r + numel, none=0.1 if numel > 1 else 0.0)
    if numel > 1:
        d["ids"][:n] = np.arange(n)
    d["ranks"] = torch.tensor([r - 1, 1, 7, 9, 0], dtype=torch.int32)
    for a, own in enumerate(d["ranks"].tolist()):
        d["A"][a, own:], d["B"][a, :, own:] = float("nan"), float("nan")
    clean = {**d, "A": d["A"].nan_to_num(0.0), "B": d["B"].nan_to_num(0.0)}
    check(clean, call(d, B), f"ranks r={r} numel={numel} K={K} B={B}")


FORMS = [(24, 2, 64, 16), (24, 2, 8200, 16), (70, 3, 264, 64), (70, 3, 264, 32)]   # rows, adapters, K, block_m


@pytest.mark.parametrize("numel,n,K,B", FORMS)
def test_infinities_stale_entries_and_strided_rows_in_both_forms(numel, n, K, B):
    d = make(numel, n, 16, 136, K, 31)
    d["ids"][5], d["ids"][6] = 0, 1
    al, _ = aligned(d["ids"].reshape(-1, 1), 0, n, B)
    end = int(al[2])
    al[0][end:] = 3                                   # entries of an earlier, longer batch
    al[1][end // B:] = 1
    base, x = strided(d["base"], 168), strided(d["x"], K + 16)
    into = torch.full((numel, 160), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (d["A"].cuda(), d["B"].cuda(), al, B, d["scales"].cuda())
    got = P.moe_adapters_add(base, x, *args, out=into[:, :136])
    check(d, got, "strided, stale")
    assert bool((into[:, 136:] == 5.0).all())
    x[5, 9], x[6, 3] = float("inf"), float("nan")     # their own rows alone
    bad = P.moe_adapters_add(base, x, *args)
    rows = [m for m in range(numel) if m not in (5, 6)]
    assert torch.equal(bad[rows], got[rows])
    assert not bool(bad[5].isfinite().any()) and bool(bad[6].isnan().all())


@pytest.mark.parametrize("numel,n,r,K,B,two", [(1, 1, 16, 8456, 16, True), (96, 6, 16, 1032, 16, False), (96, 6, 16, 4104, 16, True),
                                               (130, 3, 64, 520, 64, True), (90, 4, 200, 264, 32, True)])
def test_replayed_graphs_in_both_forms(numel, n, r, K, B, two):
    """Two graphs with a workspace each, replayed side by side; what a workspace holds before a replay is not used."""
    N = 264
    d = make(numel, n, r, N, K, 33)
    base, x, A, Bm, s = (d[key].cuda() for key in ("base", "x", "A", "B", "scales"))
    batches = [aligned(np.random.default_rng(t).integers(-1 if numel > 1 else 0, n, (numel, 1)).astype(np.int32), 0, n, B)[0]
               for t in range(4)]
    sets = []
    for i in range(2):
        al, out = tuple(t.clone() for t in batches[i]), torch.empty_like(base)
        work = torch.empty(P.adapters_workspace(numel, n, r, K, B), device="cuda")
        run = lambda al=al, out=out, work=work: P.moe_adapters_add(base, x, A, Bm, al, B, scales=s, out=out, work=work)  # noqa: E731
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        sets.append((graph, al, out, work, torch.cuda.Stream()))
    for turn in range(4):
        for i, (_, al, _, work, _) in enumerate(sets):
            for t, v in zip(al, batches[(turn + i) % 4]):
                t.copy_(v)
            work.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, _, _, _, stream in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for i, (_, _, out, work, _) in enumerate(sets):
            want = P.moe_adapters_add(base, x, A, Bm, batches[(turn + i) % 4], B, scales=s)
            assert torch.equal(out, want), (turn, i)
            assert bool(work.isnan().all()) != two    # (of two launches: the inner products went through it)


def test_two_launches_of_rows_past_four_gigabytes():
    numel, ld = 48, 1 << 26
    d = make(numel, 3, 64, 128, 264, 35)
    far = lambda t: torch.as_strided(torch.empty((numel - 1) * ld + t.shape[1], dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                                     t.shape, (ld, 1)).copy_(t.cuda())
    out = far(torch.zeros((numel, 128)))
    check(d, call(d, 16, base=far(d["base"]), x=far(d["x"]), out=out), "far rows")
    torch.cuda.empty_cache()
