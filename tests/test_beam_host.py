"""The operators of beam search over the paged cache without a GPU: the host code and the kernels' index arithmetic under
sanitizers, the refusals of the binding, the definitions themselves."""
import itertools
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle.beam_oracle as BO
import rank_adapter_gemm_build_amd as rx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "rank_adapter_gemm_build_amd", "csrc")
BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def test_host_code_and_index_arithmetic_under_asan_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if not gxx or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("g++ or the ROCm headers are missing")
    exe = str(tmp_path / "beam_sanitized")
    flags = ["address", "undefined"]
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=" + ",".join(flags),
           "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *[os.path.join(CSRC, f) for f in ("api.cpp", "beam.cpp", "shared.cpp")],
           os.path.join(HERE, "hip_stubs.cpp"), os.path.join(HERE, "beam_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-6000:])
    assert r.stdout.strip().endswith("0 failures")


def test_exported_constants():
    text = open(os.path.join(ROOT, "include", "raxlora.h")).read()
    for name in ("LORA_MAX_BEAMS", "LORA_FORK_META", "LORA_MAX_LAYERS"):
        assert re.search(rf"#define\s+{name}\s+{getattr(rx, name)}\b", text), name
    assert re.search(r"#define\s+LORA_MAX_VOCAB\s+\(1 << 24\)", text) and rx.LORA_MAX_VOCAB == 1 << 24


def test_missing_device_is_reported():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for make in (lambda: rx.Beams(0, 4, 4, 1000), lambda: rx.SharedAttention(0, 4, 8, 8, 2, 64)):
        with pytest.raises(rx.LoraError) as e:
            make()
        assert e.value.status in (rx.LORA_ERR_NO_DEVICE, rx.LORA_ERR_HIP)


# ------------------------------------------------------------------------- the binding
class _NoCalls:
    def __getattr__(self, name):
        raise AssertionError(f"the library was called: {name}")


@pytest.fixture
def no_calls(monkeypatch):
    monkeypatch.setattr(rx.beam, "lib", _NoCalls())


def _object(cls, **kw):
    o = object.__new__(cls)
    o.__dict__.update(handle=0, **kw)
    return o


def _cache(dtype=BF, pages=4):
    return rx.KVCache(torch.zeros(pages, 16, 2, 32, dtype=dtype), torch.zeros(pages, 16, 2, 32, dtype=dtype))


def _far(rows, width, dtype, stride):
    """Rows `stride` elements apart, without their memory."""
    return torch.empty_strided((rows, width), (stride, 1), dtype=dtype, device="meta")


def zeros(n, dtype=I32):
    return torch.zeros(n, dtype=dtype)


@pytest.mark.parametrize("kw", [dict(max_requests=2 ** 31), dict(beams=2 ** 32 + 4), dict(vocab=2 ** 32 + 100), dict(candidates=2 ** 32 + 4)])
def test_beam_sizes_past_31_bits_are_refused(no_calls, kw):
    with pytest.raises(ValueError, match=next(iter(kw))):
        rx.Beams(0, **{**dict(max_requests=4, beams=4, vocab=100, candidates=4), **kw})


@pytest.mark.parametrize("at", range(5))
def test_shared_sizes_past_31_bits_are_refused(no_calls, at):
    sizes = [4, 8, 4, 2, 32]
    sizes[at] += 2 ** 32
    with pytest.raises(ValueError):
        rx.SharedAttention(0, *sizes)


@pytest.mark.parametrize("change,err", [
    (dict(logits=torch.zeros(8, 100, dtype=torch.float16)), TypeError), (dict(logits=torch.zeros(8, 99)), ValueError),
    (dict(logits=torch.zeros(7, 100)), ValueError), (dict(logits=torch.zeros(800)), ValueError), (dict(logits=None), ValueError),
    (dict(logits=torch.zeros(100, 8).t()), ValueError), (dict(logits=_far(8, 100, F32, 2 ** 31)), ValueError),
    (dict(logits=torch.zeros(1, 100).expand(8, 100)), ValueError), (dict(scores=zeros(8, torch.float64)), TypeError),
    (dict(scores=zeros(7, F32)), ValueError), (dict(scores=zeros(16, F32)[::2]), ValueError), (dict(scores=None), TypeError),
    (dict(parents=zeros(5)), ValueError), (dict(parents=zeros(6, I64)), TypeError), (dict(tokens=zeros(12)[::2]), ValueError),
    (dict(tokens=[0] * 6), TypeError), (dict(scores_out=zeros(5, F32)), ValueError), (dict(scores_out=zeros((2, 3), F32)), ValueError),
    (dict(ended=zeros(7)), ValueError), (dict(ended=zeros(8, torch.bool)), TypeError), (dict(ended_out=zeros(5)), ValueError),
    (dict(weights=zeros(7, F32)), ValueError), (dict(weights=zeros(8)), TypeError), (dict(end_token=2 ** 32 + 1), ValueError),
    (dict(), ValueError),   # all well, but on the host
])
def test_beam_select_refuses(no_calls, change, err):
    a = dict(logits=torch.zeros(8, 100), scores=zeros(8, F32), parents=zeros(6), tokens=zeros(6), scores_out=zeros(6, F32),
             ended=zeros(8), ended_out=zeros(6), weights=zeros(8, F32), end_token=5)
    a.update(change)
    with pytest.raises(err):
        rx.beam_select(_object(rx.Beams, device=0, max_requests=2, beams=4, vocab=100, candidates=3), a.pop("logits"), a.pop("scores"),
                       a.pop("parents"), a.pop("tokens"), a.pop("scores_out"), **a)


@pytest.mark.parametrize("change,err", [
    (dict(parents=zeros(5)), ValueError), (dict(parents=zeros(3, I64)), TypeError), (dict(lens=zeros(2)), ValueError),
    (dict(lens=zeros(4)), ValueError), (dict(ring=zeros(7)), ValueError), (dict(ring=zeros(9)), ValueError), (dict(cursor=zeros(2)), ValueError),
    (dict(shares=zeros(9)), ValueError), (dict(shares=zeros(7)), ValueError), (dict(table=zeros((2, 4))), ValueError),
    (dict(table=zeros((4, 3)).t()), ValueError), (dict(table=_far(3, 4, I32, 2 ** 32 + 4)), ValueError), (dict(page=2 ** 32 + 16), ValueError),
    (dict(shares=None), TypeError), (dict(), ValueError),
])
def test_page_fork_refuses(no_calls, change, err):
    a = dict(parents=zeros(3), lens=zeros(3), ring=zeros(8), cursor=zeros(4), shares=zeros(8), table=zeros((3, 4)), page=16)
    a.update(change)
    plan = _object(rx.ForkPlan, device=0, max_rows=4, num_pages=8, _out=[0] * 5)
    with pytest.raises(err):
        rx.page_fork(plan, a["parents"], a["lens"], a["ring"], a["cursor"], a["shares"], a["table"], a["page"])


@pytest.mark.parametrize("rows,pages", [(-1, 8), (rx.LORA_MAX_SEQS + 1, 8), (4, 0), (4, 2 ** 31)])
def test_fork_plan_sizes(rows, pages):
    with pytest.raises(ValueError):
        rx.ForkPlan(0, rows, pages)


@pytest.mark.parametrize("change,err", [
    (dict(caches=torch.zeros(4)), TypeError), (dict(caches=[_cache()]), TypeError), (dict(src=zeros(2, I64)), TypeError),
    (dict(src=zeros(4)[::2]), ValueError), (dict(dst=zeros(1)), ValueError), (dict(dst=zeros(3)), ValueError),
    (dict(tokens=zeros(1)), ValueError), (dict(tokens=zeros(3)), ValueError), (dict(tokens=zeros(2, I64)), TypeError),
])
def test_page_copy_refuses(no_calls, change, err):
    a = dict(caches=_cache(), src=zeros(2), dst=zeros(2), tokens=zeros(2))
    a.update(change)
    with pytest.raises(err):
        rx.page_copy(a["caches"], a["src"], a["dst"], a["tokens"])


def test_page_copy_on_another_device_is_refused(no_calls):
    cache = _object(rx.KVCache, device=0, ref=None)
    with pytest.raises(ValueError, match="src"):
        rx.page_copy(cache, zeros(2), zeros(2))


def test_layers_refused():
    for bad in ([], [1], [_cache()] * (rx.LORA_MAX_LAYERS + 1), [_cache(), None]):
        with pytest.raises(ValueError):
            rx.KVLayers(bad)
    assert len(rx.KVLayers([_cache()] * rx.LORA_MAX_LAYERS).c) == rx.LORA_MAX_LAYERS


@pytest.mark.parametrize("change,err", [
    (dict(q=torch.zeros(3, 128)), TypeError), (dict(q=torch.zeros(3, 64, dtype=BF)), ValueError), (dict(q=_far(3, 128, BF, 2 ** 32 + 128)), ValueError),
    (dict(out=torch.zeros(4, 128, dtype=BF)), ValueError), (dict(out=_far(3, 128, BF, 2 ** 31)), ValueError),
    (dict(block_table=zeros((2, 4), I64)), TypeError), (dict(block_table=zeros((1, 4))), ValueError),
    (dict(block_table=_far(2, 4, I32, 2 ** 32 + 4)), ValueError), (dict(seq_lens=zeros(1)), ValueError), (dict(query_start=zeros(0)), ValueError),
    (dict(group_start=zeros(0)), ValueError), (dict(group_start=[0, 2]), TypeError), (dict(common=zeros(2)), ValueError),
    (dict(common=zeros(0)), ValueError), (dict(common=zeros(1, I64)), TypeError), (dict(lse=torch.zeros(3, 2)), ValueError),
    (dict(lse=torch.zeros(3, 4, dtype=BF)), ValueError), (dict(lse=torch.zeros(4, 3).t()), ValueError), (dict(), ValueError),
])
def test_shared_attention_refuses(no_calls, change, err):
    a = dict(q=torch.zeros(3, 128, dtype=BF), out=torch.zeros(3, 128, dtype=BF), block_table=zeros((2, 4)), seq_lens=zeros(2),
             query_start=zeros(3), group_start=zeros(2), common=zeros(1), lse=None)
    a.update(change)
    att = _object(rx.SharedAttention, device=0, num_q_heads=4, num_kv_heads=2, head_dim=32)
    with pytest.raises(err):
        rx.shared_attention(att, a["q"], _cache(), a["block_table"], a["seq_lens"], a["query_start"], a["group_start"], a["common"], a["out"],
                            lse=a["lse"])


# ------------------------------------------------------------------------- the definitions
def test_select_by_hand():
    """Two beams of a vocabulary of 3.  Beam 0: weights 1 : 2 : 1, score ln 8; beam 1 has ended with score ln 3."""
    x = [[0.0, math.log(2), 0.0], [9.0, 9.0, 9.0]]
    got = BO.select(x, [math.log(8), math.log(3)], 2, 4, ended=[0, 1], end_token=2)[0]
    want = [(0, 1, 4.0, 0), (1, 2, 3.0, 1), (0, 0, 2.0, 0), (0, 2, 2.0, 1)]      # row, token, e^score, ended
    assert [(r, t, e) for _, r, t, _, e in got] == [(r, t, e) for r, t, _, e in want]
    np.testing.assert_allclose([math.exp(s) for _, _, _, s, _ in got], [w for _, _, w, _ in want], rtol=1e-14)


def test_select_equals_a_search_over_all_sequences():
    """With as many beams as prefixes the search is exhaustive: it finds the best sequences of all."""
    rng = np.random.default_rng(2)
    V, steps, beams = 3, 3, 9
    cost = {}
    table = {p: rng.normal(size=V) for n in range(steps) for p in itertools.product(range(V), repeat=n)}
    for s in itertools.product(range(V), repeat=steps):
        cost[s] = sum(table[s[:i]][s[i]] - np.log(np.exp(table[s[:i]]).sum()) for i in range(steps))
    rows, scores = [()] * beams, [0.0] + [-math.inf] * (beams - 1)
    for _ in range(steps):
        got = BO.select([table[r] if s > -math.inf else np.zeros(V) for r, s in zip(rows, scores)], scores, beams, beams)[0]
        rows = [rows[r] + (t,) for _, r, t, _, _ in got] + [()] * (beams - len(got))
        scores = [s for _, _, _, s, _ in got] + [-math.inf] * (beams - len(got))
    best = sorted(cost, key=lambda s: -cost[s])[:beams]
    assert rows == best
    np.testing.assert_allclose(scores, [cost[s] for s in best], rtol=1e-12)


def test_select_leaves_out_what_has_no_score():
    nan, inf = math.nan, math.inf
    x = [[0.0, nan], [0.0, inf], [-inf, -inf], [-inf, 1.0], [5.0, 5.0], [5.0, 5.0]]
    got = BO.select(x, [0, 0, 0, 0, -inf, nan], 6, 6)[0]
    assert [(r, t) for _, r, t, _, _ in got] == [(3, 1)]


def test_fork_by_hand():
    """Pages of 4.  Row 0 holds pages 5, 6, 7 (10 tokens), row 1 page 2 (4 tokens), row 2 page 5 and its own 1 (6 tokens)."""
    table = [[5, 6, 7], [2, -1, -1], [5, 1, -1]]
    shares = [0, 0, 0, 0, 0, 1, 0, 0]
    ring = [3, 4, 0, -1, -1, -1, -1, -1]
    out, lens, tab, rg, cur, sh = BO.page_fork([0, 0, -1], [10, 4, 6], table, 3, ring, [0, 3], shares, 4)
    # row 0 goes on in place, row 1 shares its full pages and has its own copy of the last (page 3), rows 1's and 2's go back
    assert lens == [10, 10, 0] and tab[0].tolist() == [5, 6, 7] and tab[1].tolist() == [5, 6, 3]
    assert out["copy_src"] == [-1, 7, -1] and out["copy_dst"] == [-1, 3, -1] and out["copy_tokens"] == [0, 2, 0]
    assert sh == [0, 0, 0, 0, 0, 1, 1, 0]                      # page 5: rows 0 and 1 now, 6: shared as well
    assert cur == [1, 4] and rg[:5] == [3, 4, 0, 1, 2]
    assert out["meta"] == [1, 2, 0, 0, 4, 0, 0, 0]


@pytest.mark.parametrize("seed", range(30))
def test_fork_keeps_every_page(seed):
    """Any forks: each page is held (by shares + 1 rows) or free, once, and a row's partly filled page is its own."""
    rng = np.random.default_rng(seed)
    rows, page, cols = int(rng.integers(1, 7)), 4, 5
    pages = int(rng.integers(6, 40))
    table, lens, shares = np.full((rows, cols), -1), [0] * rows, [0] * pages
    ring, cursor = list(rng.permutation(pages)), [0, pages]
    for _ in range(12):
        parents = [int(rng.integers(-1, rows)) for _ in range(rows)]
        out, lens, table, ring, cursor, shares = BO.page_fork(parents, lens, table, cols, ring, cursor, shares, page)
        for r in range(rows):                                   # each row gains up to a page's tokens, drawing a page as a plan would
            for _ in range(int(rng.integers(0, page + 1))):
                if lens[r] == cols * page:
                    break
                if lens[r] % page == 0:
                    if cursor[1] == 0:
                        break
                    table[r, lens[r] // page] = ring[cursor[0]]
                    cursor = [(cursor[0] + 1) % pages, cursor[1] - 1]
                lens[r] += 1
        holders = np.zeros(pages, dtype=int)
        for r in range(rows):
            for c in range(-(-lens[r] // page)):
                holders[table[r, c]] += 1
        free = [ring[(cursor[0] + i) % pages] for i in range(cursor[1])]
        assert len(set(free)) == len(free) and not holders[free].any() and (holders > 0).sum() + len(free) == pages
        assert [max(0, h - 1) for h in holders] == shares
        for r in range(rows):
            if lens[r] % page:
                assert shares[table[r, lens[r] // page]] == 0
        assert out["meta"][3] == 0
