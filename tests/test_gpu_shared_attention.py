"""Shared attention on the GPU against its 64-bit definition, and against the paged attention of the same sequences."""
import numpy as np
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
import test_gpu_kv as base
from lora_cases import record_error
from test_gpu_kv import BF, CACHES, DT, F32, HALF_STEP, act_of, f64, ints, make_cache, poison_unseen

pytestmark = pytest.mark.gpu


def shared_case(seed, groups, news, hq, kv, dim, cache, order="token", page=16, pad=0, spread=1.0):
    """groups: [(common tokens, [own tokens of each member, its new ones among them])]; own = None: a sequence of length 0.
    Members of a group have its common tokens in the same pages; returns q, k, v, table, lens, starts, group_start, common."""
    rng = np.random.default_rng(seed)
    rows, lens, at = [], [], 0
    for common, own in groups:
        both = list(range(at, at + -(-common // page)))
        at += len(both)
        for x in own:
            n = common + x if x is not None else common
            rest = max(0, -(-n // page) - len(both))
            rows.append(both + list(range(at, at + rest)))
            at += rest
            lens.append(n if x is not None else 0)
    pages = at + 2
    ids = rng.permutation(pages)
    table = np.full((len(rows), max([1] + [len(r) for r in rows]) + 1), -1)
    for i, r in enumerate(rows):
        table[i, :len(r)] = ids[r]
    news = [news] * len(rows) if isinstance(news, int) else news
    T = sum(news)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    k, v = make_cache(cache, pages, page, kv, dim, order, seed + 1, pad)
    q = (torch.randn(T, hq * dim + pad, generator=g, device="cuda") * spread).to(act_of(cache))[:, :hq * dim]
    return (q, k, v, table, lens, np.concatenate([[0], np.cumsum(news)]).astype(int),
            np.concatenate([[0], np.cumsum([len(o) for _, o in groups])]).astype(int), [c for c, _ in groups])


def call(case, hq, kv, dim, scales=(1.0, 1.0), scale=None, obj=None, stream=None, lse=True, out=None):
    q, k, v, table, lens, starts, group_start, common = case
    T, pad = q.shape[0], q.stride(0) - q.shape[1] if q.shape[0] > 1 else 0
    out = torch.full((T, hq * dim + pad), 7.0, dtype=q.dtype, device="cuda")[:, :hq * dim] if out is None else out
    ls = torch.full((T, hq), 7.0, dtype=F32, device="cuda") if lse else None
    obj = obj or rx.SharedAttention(0, max(1, len(lens)), max(1, T), hq, kv, dim)
    rx.shared_attention(obj, q, rx.KVCache(k, v, *scales), ints(table), ints(lens), ints(starts), ints(group_start), ints(common), out,
                        scale=scale, lse=ls, stream=stream)
    torch.cuda.synchronize()
    return out, ls


def run(groups, news, hq, kv, dim, cache, seed=0, poison=float("nan"), page=16, order="token", pad=0, spread=1.0):
    case = shared_case(seed, groups, news, hq, kv, dim, cache, order, page, pad, spread)
    q, k, v, table, lens, starts, group_start, common = case
    if poison is not None:
        poison_unseen(k, v, table, lens, page, poison)
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    out, lse = call(case, hq, kv, dim, scales)
    # the definition: a sequence's own row names the common pages too
    base.check_attend(q, k, v, table, lens, starts, page, hq, kv, dim, out, lse, dim ** -0.5, 0, scales,
                      f"shared {len(groups)} groups, {len(lens)} seqs {hq}/{kv}x{dim} {cache}")
    again, _ = call(case, hq, kv, dim, scales, lse=False)
    assert torch.equal(out, again)                       # the same bits again, with or without lse
    return case, out, lse


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("common", [1, 15, 16, 17, 32, 100, 127, 128, 129, 640, 1000])
def test_common_lengths(common, cache):
    run([(common, [1, 5, 40])], 1, 8, 2, 64, cache, seed=common)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("own", [1, 2, 15, 16, 17, 33, 128, 300])
def test_own_lengths(own, cache):
    run([(48, [own, own, 3]), (50, [own])], 1, 4, 1, 128, cache, seed=own)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_head_dims(dim, cache):
    run([(70, [3, 20]), (200, [1, 2, 9])], 1, 4, 2, dim, cache, seed=dim)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("hq,kv", [(1, 1), (4, 4), (7, 1), (8, 2), (16, 1), (17, 1), (40, 2), (71, 1)])
@pytest.mark.parametrize("members", [1, 3, 9])
def test_head_groups(hq, kv, members, cache):
    run([(90, [1 + 7 * i for i in range(members)])], 1, hq, kv, 32, cache, seed=hq + members)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("members", [5, 16, 17, 33, 64, 65, 100])
def test_many_members(members, cache):
    """Rows of a group in one block and in several."""
    run([(300, [1 + i % 50 for i in range(members)])], 1, 8, 2, 64, cache, seed=members)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("news", [[2, 2, 2, 2], [4, 1, 7, 3], [1, 33, 5, 0], [0, 50, 1, 2], [0, 0, 0, 1]])
def test_several_new_tokens(news, cache):
    run([(64, [60, 70]), (33, [55, 8])], news, 4, 2, 64, cache, seed=sum(news))


@pytest.mark.parametrize("cache", CACHES)
def test_groups_of_all_kinds(cache):
    """Single members, nothing in common, sequences of length 0 (the first of a group among them), a common part longer than a
    member, pages of 64."""
    groups = [(100, [5]), (0, [30, 1]), (64, [None, 3, 9]), (130, [None, None]), (16, [1, None, 1]), (257, [80] * 5)]
    run(groups, 1, 8, 2, 128, cache, seed=3)
    run(groups, 1, 8, 2, 128, cache, seed=4, page=64, order="head")


@pytest.mark.parametrize("order,pad", [("token", 32), ("head", 16), ("head", 0)])
@pytest.mark.parametrize("cache", CACHES)
def test_strides(cache, order, pad):
    run([(96, [7, 30, 2]), (20, [15, 15])], 1, 8, 4, 64, cache, order=order, pad=pad, seed=9)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cache", CACHES)
def test_what_no_row_sees_has_no_effect(cache, poison):
    run([(35, [1, 4, 20]), (16, [None, 3])], 1, 8, 2, 64, cache, poison=poison, seed=5)


@pytest.mark.parametrize("cache", CACHES)
def test_wide_scores(cache):
    """Scores of some hundreds, so that one of the two results has all the weight."""
    run([(80, [40, 3]), (200, [200])], 1, 4, 2, 128, cache, spread=12.0, seed=6)


def near_paged(case, hq, kv, dim, scales, out, lse, what):
    """The paged attention's output of the same sequences, which differs by rounding: each is off by half a step of out and,
    relative to sum_j p_j |v_j| <= max |v|, by 2^-15 (16-bit) or 2^-17 (fp32, with the scores' own rounding)."""
    q, k, v, table, lens, starts, _, _ = case
    want, wl = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
    rx.paged_attention(rx.Attention(0, len(lens), q.shape[0], hq, kv, dim), q, rx.KVCache(k, v, *scales), ints(table), ints(lens), ints(starts),
                       want, lse=wl)
    torch.cuda.synchronize()
    most = float(torch.nan_to_num(v.float()).abs().max()) * scales[1]
    tol = 2 * HALF_STEP[q.dtype] * want.float().abs() + 2 * most * (2.0 ** -15 if q.dtype == BF else 2.0 ** -17)
    err = (out.float() - want.float()).abs()
    record_error(what, "of tolerance", float((err / tol).max()), 1.0)
    assert (err <= tol).all()
    assert torch.equal(lse.isneginf(), wl.isneginf())
    fine = ~wl.isneginf()
    assert ((lse - wl).abs()[fine] <= 2.0 ** -16 + wl.abs()[fine] * 2.0 ** -21).all()


LARGE = {"one-group": ([(5000, [1 + 37 * i % 700 for i in range(40)])], 1, 32, 8, 128),
         "beams": ([(800 + 391 * g, [1 + (31 * g + 7 * i) % 150 for i in range(8)]) for g in range(20)], 1, 32, 8, 128),
         "chats-and-loners": ([(3000, [50] * 64), (0, [900] * 9), (16, [5] * 30), (2000, [1500])], 1, 16, 4, 64),
         "drafts": ([(1000, [300] * 16), (500, [20] * 10)], 4, 16, 2, 128),
         "prompts": ([(700, [300, 260, 400]), (64, [200])], [250, 260, 300, 130], 8, 2, 64),
         "many": ([(64 + 16 * (g % 5), [1 + (i + g) % 40 for i in range(1 + g % 7)]) for g in range(500)], 1, 4, 1, 64),
         "wide-heads": ([(2000, [60] * 30)], 1, 8, 2, 256), "wide-blocks": ([(704, [3] * 107)], 1, 1, 1, 192),
         "wide-short-blocks": ([(64, [22] * 20)], 1, 32, 4, 256), "wide-drafts": ([(64, [22] * 5), (30, [9] * 9)], 4, 32, 4, 192),
"one-head": ([(9000, [100] * 200)], 1, 8, 1, 96)}


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("name", sorted(LARGE))
def test_large_steps_equal_the_paged_attention(name, cache):
    groups, news, hq, kv, dim = LARGE[name]
    case = shared_case(len(name), groups, news, hq, kv, dim, cache)
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    out, lse = call(case, hq, kv, dim, scales)
    near_paged(case, hq, kv, dim, scales, out, lse, f"shared against paged {name} {cache}")
    again, _ = call(case, hq, kv, dim, scales)
    assert torch.equal(out, again)


@pytest.mark.parametrize("cache", CACHES)
def test_sequences_outside_the_groups_and_partial_common_parts(cache):
    """Groups that leave out sequences at both ends; common lengths below what the members share, and above what one of them has."""
    case = list(shared_case(8, [(100, [20, 30, 1, 9]), (60, [8, 5, 50])], 1, 8, 2, 64, cache))
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    for group_start, common in (([1, 3], [77]), ([0, 0, 2, 2, 4, 7], [50, 1, 9, 96, 30]), ([4, 7], [0]), ([0], []), ([3, 4], [100])):
        case[6], case[7] = group_start, common
        out, lse = call(tuple(case), 8, 2, 64, scales)
        near_paged(tuple(case), 8, 2, 64, scales, out, lse, "partial groups")
    # a member shorter than the common part reads all its keys itself, the first of its group too
    case = list(shared_case(8, [(100, [20, 30, 1, 9])], 1, 8, 2, 64, cache))
    for short in (0, 2):
        case[4] = [120, 130, 101, 109]
        case[4][short] = 90
        out, lse = call(tuple(case), 8, 2, 64, scales)
        near_paged(tuple(case), 8, 2, 64, scales, out, lse, "a short member")


def test_nan_queries_and_keys_reach_their_rows_only():
    groups, hq, kv, dim = [(200, [9, 30, 4]), (40, [3])], 8, 2, 64
    for cache in ("bf16", "f32"):
        case = shared_case(2, groups, 1, hq, kv, dim, cache)
        want, wl = call(case, hq, kv, dim)
        q, k, v, table, *rest = case
        bad = q.clone()
        bad.view(-1, hq, dim)[1, 5, 7] = float("nan")
        got, gl = call((bad, k, v, table, *rest), hq, kv, dim)
        hit = torch.zeros(4, hq, dtype=torch.bool, device="cuda")
        hit[1, 5] = True
        assert got.view(-1, hq, dim)[hit].isnan().all() and gl[hit].isnan().all()
        assert torch.equal(got.view(-1, hq, dim)[~hit], want.view(-1, hq, dim)[~hit]) and torch.equal(gl[~hit], wl[~hit])
        # a NaN key among the common ones: every member's heads of its kv head; an own one: its sequence's
        for page_of, at, rows in ((table[0][3], 5, [0, 1, 2]), (table[1][200 // 16 + 1], 1, [1])):
            nk = k.clone()
            nk[int(page_of), at, 1, 3] = float("nan")
            got, gl = call((q, nk, v, table, *rest), hq, kv, dim)
            hit = torch.zeros(4, hq, dtype=torch.bool, device="cuda")
            hit[rows, hq // kv:] = True
            assert got.view(-1, hq, dim)[hit].isnan().all() and gl[hit].isnan().all()
            assert torch.equal(got.view(-1, hq, dim)[~hit], want.view(-1, hq, dim)[~hit])


def test_infinite_values_where_they_are_seen():
    """Values that are infinite in the common part, in the own part, and past a sequence's end."""
    groups, hq, kv, dim = [(64, [9, 30]), (64, [3])], 4, 2, 64
    for cache in ("bf16", "f32"):
        q, k, v, table, lens, *rest = shared_case(2, groups, 1, hq, kv, dim, cache)
        want, _ = call((q, k, v, table, lens, *rest), hq, kv, dim)
        v[int(table[0][1]), 3, 0, 11] = float("inf")          # common to sequences 0 and 1
        v[int(table[1][5]), 2, 1, 7] = float("-inf")          # sequence 1's own
        v[int(table[2][4]), 3:, :, :] = float("inf")          # past sequence 2's end
        got, _ = call((q, k, v, table, lens, *rest), hq, kv, dim)
        got, want = got.view(3, hq, dim), want.view(3, hq, dim)
        assert (got[:2, :2, 11] == float("inf")).all() and (got[1, 2:, 7] == float("-inf")).all()
        fine = torch.ones_like(got, dtype=torch.bool)
        fine[:2, :2, 11] = False
        fine[1, 2:, 7] = False
        assert torch.equal(got[fine], want[fine])


def test_wrong_words_stay_in_bounds():
    groups, hq, kv, dim = [(64, [9, 30]), (40, [3, 8, 1])], 4, 2, 64
    case = list(shared_case(2, groups, 1, hq, kv, dim, "bf16"))
    big = 2 ** 31 - 1
    obj = rx.SharedAttention(0, 5, 5, hq, kv, dim)
    good, _ = call(tuple(case), hq, kv, dim, obj=obj)
    for group_start, common in (([-5, 3, big], [big, -7]), ([4, 2, 5], [64, 40]), ([5, 5, 0], [1, 1]), ([0, big, -big], [10, 10]), ([0, 2, 5], [10 ** 6, -1])):
        bad = list(case)
        bad[6], bad[7] = group_start, common
        call(tuple(bad), hq, kv, dim, obj=obj)
    for lens, starts in (([big, -3, 10, 5, 0], case[5]), (case[4], [0, 3, 1, 5, 2, 9]), (case[4], [-4, 9, big, -big, 0, 1])):
        bad = list(case)
        bad[4], bad[5] = lens, starts
        call(tuple(bad), hq, kv, dim, obj=obj)
    bad = list(case)
    bad[3] = case[3].copy()
    bad[3][0, 0], bad[3][3, 1], bad[3][1, 5] = 10 ** 9, -4, k_pages(case)
    call(tuple(bad), hq, kv, dim, obj=obj)
    again, _ = call(tuple(case), hq, kv, dim, obj=obj)     # the object works on after them
    assert torch.equal(good, again)


def k_pages(case):
    return case[1].shape[0]


def test_wrong_pages_are_left_out():
    groups, hq, kv, dim = [(64, [9, 30]), (40, [3])], 4, 2, 64
    case = list(shared_case(2, groups, 1, hq, kv, dim, "f32"))
    q, k, v, table, lens, starts, group_start, common = case
    table[:2, 1] = -1                                     # a common page that is not there
    table[1, 5] = k.shape[0] + 3                          # an own one
    out, lse = call(case, hq, kv, dim)
    base.check_attend(q, k, v, table, lens, starts, 16, hq, kv, dim, out, lse, dim ** -0.5, 0, (1.0, 1.0), "shared, pages absent")


def test_rows_of_no_sequence_are_left_as_they_were():
    q, k, v, table, lens, starts, group_start, common = shared_case(2, [(64, [9, 30])], [2, 3], 4, 2, 64, "bf16")
    wide = torch.randn(9, 256, device="cuda").to(BF)
    wide[:5] = q
    out = torch.full((9, 256), 7.0, dtype=BF, device="cuda")
    got, lse = call((wide, k, v, table, lens, starts, group_start, common), 4, 2, 64, out=out)
    want, wl = call((q, k, v, table, lens, starts, group_start, common), 4, 2, 64)
    assert (got[5:] == 7).all() and (lse[5:] == 7).all() and torch.equal(got[:5], want) and torch.equal(lse[:5], wl)


def test_no_sequences_or_tokens():
    k, v = make_cache("bf16", 3, 16, 2, 64, "token", 1)
    obj = rx.SharedAttention(0, 4, 4, 4, 2, 64)
    e = torch.zeros(0, 256, dtype=BF, device="cuda")
    rx.shared_attention(obj, e, rx.KVCache(k, v), ints([[0]]), ints([]), ints([0]), ints([0]), ints([]), e)
    rx.shared_attention(obj, e, rx.KVCache(k, v), ints([[0]]), ints([5]), ints([0, 0]), ints([0, 1]), ints([3]), e)
    torch.cuda.synchronize()


def test_object_for_steps_of_different_sizes_streams_and_graphs():
    hq, kv, dim = 8, 2, 128
    sets = [[(3000, [5] * 20)], [(100, [40, 3]), (16, [1])], [(64, [700] * 30), (1000, [1] * 9)], [(0, [2000])]]
    cases = [shared_case(30 + i, g, 1, hq, kv, dim, "bf16") for i, g in enumerate(sets)]
    want = [call(c, hq, kv, dim)[0] for c in cases]
    obj = rx.SharedAttention(0, 64, 64, hq, kv, dim)
    s = torch.cuda.Stream()
    for _ in range(2):
        for c, x in zip(cases, want):
            s.wait_stream(torch.cuda.current_stream())
            out, _ = call(c, hq, kv, dim, obj=obj, stream=s)
            assert torch.equal(out, x)                     # the split depends on the step, not on the object
    args = [(q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), ints(gs), ints(cm), torch.zeros_like(q))
            for q, k, v, table, lens, starts, gs, cm in cases]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rx.shared_attention(obj, *args[0])
        rx.shared_attention(obj, *args[2])
    for rep in range(4):
        for a in args:
            a[-1].fill_(rep + 1.0)
        rx.shared_attention(obj, *args[1])
        g.replay()
        rx.shared_attention(obj, *args[3])
        torch.cuda.synchronize()
        for a, x in zip(args, want):
            assert torch.equal(a[-1], x)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_offsets_past_32_bits(cache):
    """Pages 2^27 elements apart."""
    dim, kv, page, hq = 64, 2, 16, 8
    case = shared_case(3, [(200, [60, 100])], 1, hq, kv, dim, cache)
    q, k, v, *rest = case
    pages, stride, far = k.shape[0], 1 << 27, []
    for src in (k, v):
        flat = torch.empty((pages - 1) * stride + page * kv * dim, dtype=DT[cache], device="cuda")
        x = flat.as_strided((pages, page, kv, dim), (stride, kv * dim, dim, 1))
        (x.view(torch.uint8) if cache == "fp8" else x).copy_(src.view(torch.uint8) if cache == "fp8" else src)
        far.append(x)
    want, _ = call(case, hq, kv, dim)
    got, _ = call((q, *far, *rest), hq, kv, dim)
    assert torch.equal(got, want) and got.any()


def test_timing_names_both_launches():
    rx.lora_timing_enable(True)
    try:
        rx.lora_timing_report()
        call(shared_case(1, [(20, [3, 4])], 1, 4, 2, 64, "bf16"), 4, 2, 64)
        rep = rx.lora_timing_report()
    finally:
        rx.lora_timing_enable(False)
    assert rep["shared_attention"][1] == 1 and rep["shared_merge"][1] == 1
