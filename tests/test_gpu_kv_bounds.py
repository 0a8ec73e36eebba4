"""What the paged-cache calls write, and nothing beside it: outputs between margins, wrong words taken at their
bounds, and the largest number of sequences in every launch shape."""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
import rank_adapter_gemm_build_amd as rx
from test_gpu_kv import CACHES, DT, act_of, attend_case, check_attend, f64, ints, run_attend

pytestmark = pytest.mark.gpu

MARGIN = 64


class Framed:
    """A tensor of `shape` inside a larger one filled with `mark`; `frame_kept` compares all around it."""

    def __init__(self, shape, dtype, mark):
        self.whole = torch.full([n + 2 * MARGIN for n in shape], mark, dtype=dtype, device="cuda")
        self.inner = self.whole[tuple(slice(MARGIN, MARGIN + n) for n in shape)]
        self.mark = mark

    def frame_kept(self):
        rest = self.whole.clone()
        rest[tuple(slice(MARGIN, MARGIN + n) for n in self.inner.shape)] = self.mark
        return bool((rest == self.mark).all())


# =============================================================================== page plan
def plan_between_margins(past, new, table, max_pages, ring, cursor, page, num_tokens):
    """The call's outputs, every vector between margins of -77."""
    R = len(past)
    v = {k: Framed([n], torch.int32, -77) for k, n in dict(past=R, new=R, ring=len(ring), cursor=4, cursor_out=2, seq_lens=R,
                                                           query_start=R + 1, positions=num_tokens, slots=num_tokens, meta=8).items()}
    tab = Framed([R, max_pages], torch.int32, -77)
    for k, x in (("past", past), ("new", new), ("ring", ring), ("cursor", list(cursor) + [0, 0])):
        v[k].inner.copy_(ints(x))
    tab.inner.copy_(ints(np.asarray(table)[:, :max_pages]))
    p = {k: f.inner.data_ptr() for k, f in v.items()}
    rx.kv._check(rx.lib.lora_page_plan(0, p["past"], p["new"], R, num_tokens, page, len(ring), p["ring"], p["cursor"], p["cursor_out"],
                                       tab.inner.data_ptr(), tab.inner.stride(0), max_pages, p["seq_lens"], p["query_start"],
                                       p["positions"], p["slots"], p["meta"], torch.cuda.current_stream().cuda_stream or None), "plan")
    torch.cuda.synchronize()
    assert all(f.frame_kept() for f in v.values()) and tab.frame_kept()
    assert v["cursor"].inner.tolist() == list(cursor) + [0, 0]
    return {k: f.inner.cpu().numpy() for k, f in v.items()}, tab.inner.cpu().numpy()


@pytest.mark.parametrize("cursor", [[-13, 5], [6, 10 ** 9], [-(2 ** 31), -1], [2 ** 31 - 1, 2 ** 31 - 1], [7, 0]])
@pytest.mark.parametrize("seqs", [8, 300])
def test_plan_with_wrong_words_writes_its_outputs_only(seqs, cursor):
    """Lengths out of range, foreign page ids and a cursor outside the ring, against the definition with the cursor's
    words at their bounds; one workgroup and several."""
    rng = np.random.default_rng(seqs)
    past, new = rng.integers(0, 60, seqs), rng.integers(-1, 20, seqs)
    past[::7], new[1::9], past[3::11] = -1, -2, 70
    table = rng.integers(-3, 40, (seqs, 4))
    table[::5, 0], table[1::6, 2] = 10 ** 9, -(2 ** 31)
    ring = rng.integers(-2, 40, 33)
    tokens = int(np.where((past >= 0) & (new > 0), new, 0).sum())
    for T in (tokens, max(1, tokens // 2), tokens + 70):
        got, tab = plan_between_margins(past, new, table, 4, ring, cursor, 16, T)
        want, wtab, wring, wcur = KO.page_plan(past, new, table, 4, ring, cursor, 16, T)
        assert got["seq_lens"].tolist() == want["seq_lens"] and got["query_start"].tolist() == want["query_start"]
        assert got["slots"].tolist() == want["slots"] and got["positions"].tolist() == want["positions"]
        assert got["meta"].tolist() == want["meta"] and got["cursor_out"].tolist() == wcur
        np.testing.assert_array_equal(tab, wtab)
        np.testing.assert_array_equal(got["ring"], wring)


def test_plan_counts_only_pages_that_were_drawn():
    """Request 0 starts a page and there is none; request 1 fits its last page and is granted: the ring stays."""
    got, tab = plan_between_margins([16, 5], [1, 1], [[2, -1], [0, -1]], 2, [1, 3, 1, 3], [3, 0], 16, 2)
    assert got["seq_lens"].tolist() == [0, 6] and got["slots"].tolist() == [-1, 5] and got["positions"].tolist() == [16, 5]
    assert got["cursor_out"].tolist() == [3, 0] and got["meta"].tolist() == [2, 0, 0, 1, 0, 0, 0, 0]
    assert tab.tolist() == [[2, -1], [0, -1]] and got["ring"].tolist() == [1, 3, 1, 3]


# =============================================================================== rotary append
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("rot", [64, 22])
@pytest.mark.parametrize("T", [1, 19, 1100])
def test_append_with_wrong_slots_writes_its_rows_and_cells_only(T, rot, cache):
    hq, kv, dim, page = 4, 2, 64, 16
    act, pages = act_of(cache), T // page + 2
    q = Framed([T, hq * dim], act, 7.0)
    k, v = (torch.full((pages + 2, page, kv, dim), 3.0, device="cuda").to(DT[cache]) for _ in "kv")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    qkv = torch.randn(T, (hq + 2 * kv) * dim, generator=g, device="cuda").to(act)
    slots = np.random.default_rng(T).permutation(pages * page)[:T].astype(np.int64)
    slots[::3] = np.resize([-1, pages * page, 2 ** 31 - 1, -(2 ** 31), pages * page + 5], len(slots[::3]))
    rx.rotary_append(rx.Rotary(0, rot, rx.rotary_frequencies(rot)), qkv, hq, ints(range(T)), ints(slots), q.inner,
                     rx.KVCache(k[1:-1], v[1:-1]))
    torch.cuda.synchronize()
    assert q.frame_kept() and not (q.inner == 7.0).all(1).any()
    kept = np.ones(((pages + 2) * page,), dtype=bool)
    kept[page + slots[(slots >= 0) & (slots < pages * page)]] = False
    for x in (k, v):
        x = f64(x).reshape(-1, kv * dim)
        assert (x[kept] == 3.0).all() and not (x[~kept] == 3.0).all(1).any()


# =============================================================================== attention
WRONG = [([5, 2, 9], [50, 60]), ([-4, 3, 2 ** 31 - 1], [2 ** 31 - 1, -5]), ([0, 7, 0], [50, 60]),
         ([2 ** 31 - 1, -(2 ** 31), 4], [10 ** 6, 60]), ([3, 3, 3], [50, 60]), ([-(2 ** 31), 2, 2], [3, 60]), ([1, 6, 5], [7, 2 ** 31 - 1])]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("starts,lens", WRONG)
@pytest.mark.parametrize("window", [0, 9])
def test_attention_with_wrong_starts_and_lengths_writes_its_rows_only(starts, lens, window, cache):
    """Starts and lengths count as the nearer bound; rows of no sequence and all around the outputs stay."""
    hq, kv, dim, page, T = 4, 2, 64, 16, 7
    q, k, v, table, _ = attend_case(5, [50, 60], [3, 4], hq, kv, dim, cache, "token")
    att = rx.Attention(0, 2, T, hq, kv, dim)
    out, lse = Framed([T, hq * dim], act_of(cache), 7.0), torch.full((T + 2 * MARGIN, hq), 7.0, device="cuda")
    for _ in range(2):                        # what wrong words leave in the object's counters would show in the second call
        rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), out.inner, window=window,
                           lse=lse[MARGIN:MARGIN + T])
    torch.cuda.synchronize()
    assert out.frame_kept() and (lse[:MARGIN] == 7).all() and (lse[MARGIN + T:] == 7).all()
    s = np.clip(starts, 0, T)
    n = np.clip(lens, 0, table.shape[1] * page)
    rows = np.zeros(T, dtype=bool)
    for r in range(2):
        rows[s[r]:s[r + 1]] = True
    left = torch.from_numpy(~rows).cuda()
    assert (out.inner[left] == 7).all() and (lse[MARGIN:MARGIN + T][left] == 7).all()
    o, ln = out.inner.clone(), lse[MARGIN:MARGIN + T].clone()
    o[left], ln[left] = 0.0, -float("inf")    # as the definition has rows of no sequence
    check_attend(q, k, v, table, n.tolist(), s, page, hq, kv, dim, o, ln, dim ** -0.5, window, (1.0, 1.0), f"starts {starts}")


# 4096 sequences: (query heads, kv heads, longest sequence)
MOST = {"one wave": (1, 1, 40), "one wave cut": (2, 2, 600), "16 rows": (3, 1, 700), "32 rows": (20, 1, 60), "64 rows": (40, 1, 60)}


@pytest.mark.parametrize("dim,cache", [(64, "bf16"), (128, "bf16"), (128, "fp8"), (256, "bf16"), (128, "f32")])
@pytest.mark.parametrize("shape", list(MOST))
def test_attention_of_the_most_sequences(shape, dim, cache):
    hq, kv, longest = MOST[shape]
    lens = np.random.default_rng(dim).integers(0, 24, rx.LORA_MAX_SEQS)
    lens[[7, 4000]] = longest, longest // 2
    run_attend(lens.tolist(), [1] * rx.LORA_MAX_SEQS, hq, kv, dim, cache, seed=dim)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_page_that_no_sequence_holds_has_no_effect_through_wrong_ids(page, dim, cache):
    """Ids outside the cache leave their keys out, whatever lies in the cache's first page."""
    lens, news, hq, kv = [6 * page - 3, 700, 40], [1, 2, 1], 4, 2
    q, k, v, table, starts = attend_case(2, lens, news, hq, kv, dim, cache, "token", page)
    for r in range(3):
        for j in range(-(-lens[r] // page)):
            if table[r][j] == 0:
                table[r][j] = -9              # the first page is held by none
    table[0][1], table[0][4], table[1][0], table[1][7] = -1, 10 ** 9, -(2 ** 31), k.shape[0]
    two = []
    for _ in range(2):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[0], hq, device="cuda")
        rx.paged_attention(rx.Attention(0, 3, q.shape[0], hq, kv, dim), q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts),
                           out, lse=lse)
        two.append((out, lse))
        for x in (k, v):
            (x.view(torch.uint8) if cache == "fp8" else x)[0] = 0x7F if cache == "fp8" else float("nan")
    assert torch.isfinite(two[0][0].float()).all() and all(torch.equal(a, b) for a, b in zip(*two))
