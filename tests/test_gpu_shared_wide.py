"""Shared attention on the GPU where groups have many rows (more than 64 a kv head), and at the ends of its ranges."""
import numpy as np
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
import test_gpu_kv as base
from test_gpu_kv import BF, F32, ints, poison_unseen
from test_gpu_shared_attention import call, near_paged, shared_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("common", [1, 63, 64, 65, 200, 513, 1999])
@pytest.mark.parametrize("members", [17, 40, 65])
def test_common_lengths_and_rows(members, common, dim, cache):
    """Rows and keys that end inside a block, a tile and a page; what no row sees is NaN."""
    case = shared_case(common + members, [(common, [1 + i % 9 for i in range(members)])], 1, 8, 2, dim, cache)
    q, k, v, table, lens, starts, _, _ = case
    poison_unseen(k, v, table, lens, 16, float("nan"))
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    out, lse = call(case, 8, 2, dim, scales)
    base.check_attend(q, k, v, table, lens, starts, 16, 8, 2, dim, out, lse, dim ** -0.5, 0, scales, f"wide {members}x{common} {dim} {cache}")
    assert torch.equal(out, call(case, 8, 2, dim, scales, lse=False)[0])


@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.125, 0.5])
@pytest.mark.parametrize("members", [3, 40])
def test_scales(members, scale, cache):
    case = shared_case(members, [(150, [1 + i % 30 for i in range(members)])], 1, 8, 2, 64, cache)
    q, k, v, table, lens, starts, _, _ = case
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    out, lse = call(case, 8, 2, 64, scales, scale=scale)
    base.check_attend(q, k, v, table, lens, starts, 16, 8, 2, 64, out, lse, scale, 0, scales, f"scale {scale} {cache}")


@pytest.mark.parametrize("members", [3, 40])
def test_common_keys_whose_scores_are_all_minus_infinity(members):
    """The common part then has no weight, and the own part all of it."""
    for cache in ("bf16", "f32"):
        case = shared_case(4, [(200, [5 + i % 30 for i in range(members)])], 1, 8, 2, 64, cache)
        q, k, v, table, *_ = case
        q.view(members, 8, 64)[:, :, 0] = 1.0
        for c in range(200 // 16):
            k[int(table[0][c]), :, :, 0] = -float("inf")
        k[int(table[0][200 // 16]), :200 % 16, :, 0] = -float("inf")
        out, lse = call(case, 8, 2, 64)
        assert out.isfinite().all() and lse.isfinite().all()
        near_paged(case, 8, 2, 64, (1.0, 1.0), out, lse, f"common part of no weight {cache}")


def test_rows_of_nan_and_values_of_infinity():
    case = shared_case(6, [(300, [4] * 40)], 1, 8, 2, 128, "bf16")
    q, k, v, table, *_ = case
    want, _ = call(case, 8, 2, 128)
    q.view(40, 8, 128)[17, 5, 3] = float("nan")
    v[int(table[0][7]), 2, 0, 90] = float("inf")
    got, _ = call(case, 8, 2, 128)
    got, want = got.view(40, 8, 128), want.view(40, 8, 128)
    assert got[17, 5].isnan().all() and (got[:, :4, 90] == float("inf")).all()
    fine = torch.ones_like(got, dtype=torch.bool)
    fine[17, 5], fine[:, :4, 90] = False, False
    assert torch.equal(got[fine], want[fine])


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_pages_that_are_not_there(cache):
    case = shared_case(6, [(300, [4 + i for i in range(40)]), (100, [20] * 3)], 1, 8, 2, 128, cache)
    q, k, v, table, lens, starts, _, _ = case
    poison_unseen(k, v, table, lens, 16, float("nan"))
    table[:40, 3], table[:40, 18], table[40:, 0] = -1, k.shape[0], 10 ** 9
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    out, lse = call(case, 8, 2, 128, scales)
    base.check_attend(q, k, v, table, lens, starts, 16, 8, 2, 128, out, lse, 128 ** -0.5, 0, scales, f"wide, pages absent {cache}")
    table[:40, :18] = -1                                  # no common key at all
    out, lse = call(case, 8, 2, 128, scales)
    base.check_attend(q, k, v, table, lens, starts, 16, 8, 2, 128, out, lse, 128 ** -0.5, 0, scales, f"wide, all pages absent {cache}")


def test_wrong_words_stay_in_bounds():
    hq, kv, dim, big = 8, 2, 64, 2 ** 31 - 1
    case = list(shared_case(2, [(300, [9] * 30), (40, [3] * 30)], 1, hq, kv, dim, "bf16"))
    obj = rx.SharedAttention(0, 60, 60, hq, kv, dim)
    good, _ = call(tuple(case), hq, kv, dim, obj=obj)
    rng = np.random.default_rng(0)
    for group_start, common in (([-5, 30, big], [big, -7]), ([40, 2, 50], [64, 40]), ([60, 60, 0], [1, 1]), ([0, big, -big], [300, 300])):
        bad = list(case)
        bad[6], bad[7] = group_start, common
        call(tuple(bad), hq, kv, dim, obj=obj)
    for starts in (rng.permutation(61), rng.integers(-big, big, 61), np.full(61, 30), np.arange(60, -1, -1)):
        bad = list(case)
        bad[5] = starts
        call(tuple(bad), hq, kv, dim, obj=obj)
    bad = list(case)
    bad[4] = rng.integers(-5, 400, 60)
    call(tuple(bad), hq, kv, dim, obj=obj)
    again, _ = call(tuple(case), hq, kv, dim, obj=obj)    # the object works on after them
    assert torch.equal(good, again)


def test_tables_for_the_longest_sequences():
    """Tables of 2^31 - 1024 tokens: a step of the lines is then more than one tile."""
    hq, kv, dim, page = 64, 16, 64, 1024
    for news, groups in ((20, [(5000, [40, 3000])]), (1, [(3000, [40, 1500, 1] * 7), (2050, [1000])])):
        case = list(shared_case(7, groups, news, hq, kv, dim, "bf16", page=page))
        table = torch.full((len(case[4]), (1 << 21) - 1), -1, dtype=torch.int32)
        table[:, :case[3].shape[1]] = torch.from_numpy(case[3].astype(np.int32))
        case[3] = table
        out, lse = call(tuple(case), hq, kv, dim)
        near_paged(tuple(case), hq, kv, dim, (1.0, 1.0), out, lse, "longest tables")


@pytest.mark.parametrize("news", [1, 17])
def test_as_many_sequences_and_groups_as_there_may_be(news):
    S = rx.LORA_MAX_SEQS
    case = list(shared_case(8, [(16 + i % 5, [news + i % 7]) for i in range(S)], news, 4, 1, 64, "bf16"))
    out, lse = call(tuple(case), 4, 1, 64)
    near_paged(tuple(case), 4, 1, 64, (1.0, 1.0), out, lse, f"{S} groups")
    case = shared_case(9, [(40, [news + i % 7 for i in range(S)])], news, 4, 1, 64, "bf16")
    out, lse = call(case, 4, 1, 64)
    near_paged(case, 4, 1, 64, (1.0, 1.0), out, lse, f"one group of {S}")


def test_two_objects_on_two_streams_and_replayed_graphs():
    hq, kv, dim = 8, 2, 128
    cases = [shared_case(40 + i, g, 1, hq, kv, dim, "bf16") for i, g in
             enumerate([[(6000, [5] * 70)], [(900, [300 + i for i in range(90)])], [(3000, [50] * 20), (100, [2] * 30)]])]
    want = [call(c, hq, kv, dim) for c in cases]
    args = [[(q, rx.KVCache(k, v), ints(t), ints(n), ints(s), ints(gs), ints(cm), torch.zeros_like(q)) for q, k, v, t, n, s, gs, cm in cases]
            for _ in "ab"]
    objs, streams = [rx.SharedAttention(0, 96, 96, hq, kv, dim) for _ in "ab"], [torch.cuda.Stream() for _ in "ab"]
    torch.cuda.synchronize()
    for _ in range(5):
        for obj, s, a in zip(objs, streams, args):
            for x in a:
                rx.shared_attention(obj, *x, stream=s)
    torch.cuda.synchronize()
    for a in args:
        for x, (w, _) in zip(a, want):
            assert torch.equal(x[-1], w)
    graphs = []
    for obj, a in zip(objs, args):
        lse = [torch.zeros(x[0].shape[0], hq, dtype=F32, device="cuda") for x in a]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for x, l in zip(a, lse):
                rx.shared_attention(obj, *x, lse=l)
        graphs.append((g, lse))
    for rep in range(3):
        for a in args:
            for x in a:
                x[-1].fill_(rep + 1.0)
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):            # at the same time
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, (_, lse) in zip(args, graphs):
            for x, l, (w, wl) in zip(a, lse, want):
                assert torch.equal(x[-1], w) and torch.equal(l, wl)


def test_a_step_of_the_lines_equals_another_split():
    """The same sequences as one group and as groups of their own differ by rounding only."""
    hq, kv, dim = 8, 2, 64
    case = list(shared_case(11, [(700, [30] * 48)], 1, hq, kv, dim, "bf16"))
    for starts in ([0, 48], [0, 24, 48], list(range(49)), [0, 17, 40]):
        case[6], case[7] = starts, [700 - i % 3 for i in range(len(starts) - 1)]
        out, lse = call(tuple(case), hq, kv, dim)
        near_paged(tuple(case), hq, kv, dim, (1.0, 1.0), out, lse, f"{len(starts) - 1} groups")
        assert out.dtype is BF


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_many_wide_groups(cache):
    """More groups than have even parts, so that shares begin and end anywhere in a unit; and as many as there may be."""
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    for groups, news, hq, kv, dim in (([(100 + 97 * g, [1 + (7 * g + i) % 40 for i in range(70)]) for g in range(24)], 1, 4, 1, 64),
                                      ([(1 + 211 * g % 1500, [1 + i % 3 for i in range(66 + g)]) for g in range(17)], 1, 8, 2, 128),
                                      ([(16 + g % 90, [70 + g % 5] * 2) for g in range(1024)], 35, 4, 1, 64)):
        case = shared_case(len(groups), groups, news, hq, kv, dim, cache)
        out, lse = call(case, hq, kv, dim, scales)
        near_paged(case, hq, kv, dim, scales, out, lse, f"{len(groups)} wide groups {cache}")
        assert torch.equal(out, call(case, hq, kv, dim, scales, lse=False)[0])
