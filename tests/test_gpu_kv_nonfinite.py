"""Paged attention where scores are not finite: a NaN query, NaN keys and scores of minus
infinity give the same whether one workgroup takes a sequence or several share it."""
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
from test_gpu_kv import CACHES, E4M3, attend_case, ints

pytestmark = pytest.mark.gpu

# lengths that one wave, one workgroup, two to eight of them and more than eight take
LENGTHS = [1, 20, 100, 300, 777, 5000]


def attend(q, k, v, table, lens, starts, hq, kv, dim, scale=None):
    out = torch.full_like(q, 7.0)
    lse = torch.full((q.shape[0], hq), 7.0, device="cuda")
    rx.paged_attention(rx.Attention(0, len(lens), q.shape[0], hq, kv, dim), q, rx.KVCache(k, v), ints(table), ints(lens),
                       ints(starts), out, scale=scale, lse=lse)
    torch.cuda.synchronize()
    return out.view(-1, hq, dim), lse


def put(cells, at, value):
    """`value` at an index of cells (an e4m3 cache has NaN only)."""
    if cells.dtype == E4M3:
        cells.view(torch.uint8)[at] = 0x7F
    else:
        cells[at] = value


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check_rows(got, want, hit):
    """Rows of `hit` [tokens, heads] are NaN in both outputs; the others keep their bits."""
    for x, y in zip(got, want):
        assert torch.isfinite(y).all()
        assert torch.isnan(x[hit]).all()
        assert same(x[~hit], y[~hit])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [64, 128, 192])
@pytest.mark.parametrize("n", LENGTHS)
def test_nan_query_gives_nan_and_no_other_row_changes(n, dim, cache):
    lens, news, hq, kv = [n], [min(n, 3)], 8, 2
    q, k, v, table, starts = attend_case(n, lens, news, hq, kv, dim, cache, "token")
    want = attend(q, k, v, table, lens, starts, hq, kv, dim)
    bad = q.clone()
    bad.view(-1, hq, dim)[news[0] - 1, 5, 7] = float("nan")
    hit = torch.zeros(news[0], hq, dtype=torch.bool, device="cuda")
    hit[news[0] - 1, 5] = True
    check_rows(attend(bad, k, v, table, lens, starts, hq, kv, dim), want, hit)


# launch shapes: one-wave workgroups uncut and cut, blocks of 16, 32 and 64 rows
SHAPES = {"one-wave": ([60 + i % 300 for i in range(256)], 1, 4, 4), "one-wave-cut": ([40 + i % 90 for i in range(600)], 1, 4, 4),
          "16-rows": ([100 + 7 * i for i in range(40)], 2, 8, 4), "32-rows": ([150 + 9 * i for i in range(32)], 3, 32, 4),
          "64-rows": ([100 + 5 * i for i in range(64)], 7, 32, 4)}


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_nan_queries_in_every_launch_shape(shape, cache):
    lens, new, hq, kv = SHAPES[shape]
    q, k, v, table, starts = attend_case(3, lens, [new] * len(lens), hq, kv, 64, cache, "token")
    want = attend(q, k, v, table, lens, starts, hq, kv, 64)
    bad, hit = q.clone(), torch.zeros(q.shape[0], hq, dtype=torch.bool, device="cuda")
    for r in range(0, len(lens), 3):
        t, h = starts[r] + r % new, r % hq
        bad.view(-1, hq, 64)[t, h, r % 64] = float("nan")
        hit[t, h] = True
    check_rows(attend(bad, k, v, table, lens, starts, hq, kv, 64), want, hit)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("n,lo,hi", [(20, 0, 16), (100, 32, 64), (100, 0, 100), (300, 128, 256), (777, 0, 128), (777, 256, 512),
                                     (777, 640, 777), (5000, 4096, 4224), (5000, 0, 2048), (5000, 0, 5000)])
def test_nan_keys_over_a_whole_part_reach_the_rows_that_see_them(n, lo, hi, cache):
    """Keys lo..hi of the first kv head: its rows are NaN, those of the second keep their bits."""
    lens, news, hq, kv, dim = [n], [2], 8, 2, 64
    q, k, v, table, starts = attend_case(n + lo, lens, news, hq, kv, dim, cache, "token")
    want = attend(q, k, v, table, lens, starts, hq, kv, dim)
    k = k.clone()
    for j in range(lo, hi):
        put(k, (table[0][j // 16], j % 16, 0), float("nan"))
    hit = torch.zeros(2, hq, dtype=torch.bool, device="cuda")
    hit[:, :hq // kv] = True
    check_rows(attend(q, k, v, table, lens, starts, hq, kv, dim), want, hit)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("n", LENGTHS)
def test_scores_of_minus_infinity_everywhere_count_as_nothing_seen(n, cache):
    """Every weight is 0: zeros and a log sum of minus infinity, as for a row that sees no key."""
    q, k, v, table, starts = attend_case(n, [n], [1], 4, 2, 64, cache, "token")
    q[:, :64] = 0.0
    q[:, 3] = 1.0
    want = attend(q, k, v, table, [n], starts, 4, 2, 64)
    k = k.clone()
    k[:, :, 0, 3] = -float("inf")
    q[:, 64:128] = 0.0
    q[:, 64 + 3] = 2.0
    out, lse = attend(q, k, v, table, [n], starts, 4, 2, 64)
    assert (out[:, :2] == 0).all() and torch.isneginf(lse[:, :2]).all()
    assert same(out[:, 2:], want[0][:, 2:]) and same(lse[:, 2:], want[1][:, 2:])
