"""Launch shapes of the paged attention that only larger batches take (one-wave workgroups,
row blocks of 32 and 64), and the operators together in the serving example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
from test_gpu_kv import CACHES, attend_case, ints, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("window", [0, 7])
def test_one_wave_workgroups(dim, window, cache):
    """1024 units or more, short rows in the table: a wave a workgroup."""
    rng = np.random.default_rng(dim)
    lens = rng.integers(0, 70, 256)
    lens[:3] = [0, 1, 200]
    run_attend(lens.tolist(), [1] * 256, 4, 4, dim, cache, seed=dim, window=window)


@pytest.mark.parametrize("cache", CACHES)
def test_one_wave_workgroups_with_several_rows(cache):
    rng = np.random.default_rng(1)
    lens = rng.integers(3, 40, 257)
    lens[5] = 900
    run_attend(lens.tolist(), rng.integers(0, 4, 257).tolist(), 8, 4, 64, cache, seed=3)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [48, 128, 256])
@pytest.mark.parametrize("hq,news,window", [(32, 3, 0), (20, 5, 0), (20, 5, 11), (24, 4, 0)])
def test_blocks_of_32_rows(dim, hq, news, window, cache):
    """32 sequences of 4 kv heads: 17 to 32 rows each."""
    rng = np.random.default_rng(dim + hq)
    lens = rng.integers(0, 90, 32)
    lens[:2] = [2, 700]
    run_attend(lens.tolist(), [news] * 32, hq, 4, dim, cache, seed=dim, window=window)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [48, 128, 256])
@pytest.mark.parametrize("hq,news,window", [(32, 7, 0), (16, 9, 0), (16, 17, 9), (8, 40, 0)])
def test_blocks_of_64_rows(dim, hq, news, window, cache):
    """64 sequences of 4 kv heads: more than 32 rows each, some of them in two blocks."""
    rng = np.random.default_rng(dim + hq)
    lens = rng.integers(0, 70, 64)
    lens[:2] = [2, 500]
    counts = np.full(64, news)
    counts[3], counts[4] = 1, 2 * news
    run_attend(lens.tolist(), counts.tolist(), hq, 4, dim, cache, seed=dim, window=window)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("kv,hq,news", [(4, 4, 1), (4, 32, 3), (4, 32, 7)])
def test_prompts(kv, hq, news, cache):
    """A long prompt beside decode tokens, in every shape of workgroup."""
    lens = [130] + [20] * 63
    run_attend(lens, [100] + [news] * 63, hq, kv, 64, cache, seed=9)
    run_attend(lens, [100] + [news] * 63, hq, kv, 64, cache, seed=9, window=33)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("hq,news", [(4, 2), (32, 3), (32, 7)])
def test_rows_that_do_not_see_a_bad_cell(hq, news, cache, bad):
    """The last cached key of every sequence holds one cell that is not finite, which only the last new token sees."""
    seqs, kv, dim = 64, 4, 64
    lens = [30 + i for i in range(seqs)]
    q, k, v, table, starts = attend_case(5, lens, [news] * seqs, hq, kv, dim, cache, "token")
    clean = v.clone()
    for r, n in enumerate(lens):
        v[table[r][(n - 1) // 16], (n - 1) % 16, :, 10] = bad
    att = rx.Attention(0, seqs, seqs * news, hq, kv, dim)
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), out)
    rx.paged_attention(att, q, rx.KVCache(k, clean), ints(table), ints(lens), ints(starts), want)
    out, want = (x.view(seqs, news, hq, dim) for x in (out, want))
    assert torch.equal(out[:, :-1], want[:, :-1])
    other = [d for d in range(dim) if d != 10]
    assert torch.equal(out[:, -1][..., other], want[:, -1][..., other])
    hit = out[:, -1, :, 10].float()
    assert torch.isnan(hit).all() if bad != bad else ((hit == bad) | torch.isnan(hit)).all()


def test_an_infinite_value_that_all_rows_see_is_kept():
    q, k, v, table, starts = attend_case(5, [200], [1], 4, 1, 64, "bf16", "token")
    v[table[0][2], 3, 0, 7], v[table[0][9], 1, 0, 8] = float("inf"), -float("inf")
    out = torch.zeros_like(q)
    rx.paged_attention(rx.Attention(0, 1, 1, 4, 1, 64), q, rx.KVCache(k, v), ints(table), ints([200]), ints(starts), out)
    out = out.view(4, 64).float()
    assert (out[:, 7] == float("inf")).all() and (out[:, 8] == -float("inf")).all()
    assert torch.isfinite(out[:, [d for d in range(64) if d not in (7, 8)]]).all()


def test_object_made_for_less_is_refused_and_for_more_gives_the_same_bits():
    lens, news = [100, 400, 3], [2, 1, 1]
    q, k, v, table, starts = attend_case(5, lens, news, 8, 2, 128, "bf16", "token")
    args = (q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts))
    outs = []
    for seqs, tokens in ((3, 4), (300, 4), (3, 5000)):
        outs.append(torch.zeros_like(q))
        rx.paged_attention(rx.Attention(0, seqs, tokens, 8, 2, 128), *args, outs[-1])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for seqs, tokens in ((2, 4), (3, 3)):
        with pytest.raises(rx.LoraError) as e:
            rx.paged_attention(rx.Attention(0, seqs, tokens, 8, 2, 128), *args, torch.zeros_like(q))
        assert e.value.status == rx.LORA_ERR_CAPACITY


def test_serving_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_serving.py")
    spec = importlib.util.spec_from_file_location("paged_serving", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # bf16 rounds the packed rows, the turned rows, the attention output and the result, 2^-9 of a
    # value each at most, and their errors add along a path of four products: 2^-5 in all is ample
    assert example.main() <= 2.0 ** -5
