"""The paged-cache operators on the GPU against their 64-bit definitions (oracle/kv_oracle.py)."""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
import rank_adapter_gemm_build_amd as rx
from lora_cases import record_error

pytestmark = pytest.mark.gpu

I32, BF, F32, E4M3 = torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn
DT = {"bf16": BF, "f32": F32, "fp8": E4M3}
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}      # largest rounding, relative to the value


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


def f64(t):
    return t.detach().float().double().cpu().numpy() if t.dtype != F32 else t.detach().double().cpu().numpy()


def act_of(cache):
    return F32 if cache == "f32" else BF


# =============================================================================== page plan
def run_plan(past, new, table, max_pages, ring, cursor, page, num_tokens, in_place=False, stream=None):
    plan = rx.PagePlan(0, max(1, len(past)), max(1, num_tokens))
    for t in (plan.seq_lens, plan.query_start, plan.positions, plan.slots, plan.meta):
        t.fill_(-77)
    tab, rg, cur = ints(table).reshape(np.asarray(table).shape), ints(ring), ints(list(cursor) + [0, 0])
    out = None if in_place else ints([-5, -5, -5, -5])
    rx.page_plan(plan, ints(past), ints(new), num_tokens, rg, cur, tab[:, :max_pages], page, cursor_out=out, stream=stream)
    torch.cuda.synchronize()
    n = len(past)
    got = {"seq_lens": plan.seq_lens[:n], "query_start": plan.query_start[:n + 1], "positions": plan.positions[:num_tokens],
           "slots": plan.slots[:num_tokens], "meta": plan.meta}
    got = {k: v.cpu().numpy().tolist() for k, v in got.items()}
    assert cur[2:].tolist() == [0, 0]              # scratch words back to zero
    if out is not None:
        assert cur[:2].tolist() == list(cursor) and out[2:].tolist() == [-5, -5]
    return got, tab.cpu().numpy(), rg.cpu().numpy(), (cur if in_place else out)[:2].tolist()


def check_plan(past, new, table, max_pages, ring, cursor, page, num_tokens, **kw):
    got, tab, rg, cur = run_plan(past, new, table, max_pages, ring, cursor, page, num_tokens, **kw)
    want, wtab, wrg, wcur = KO.page_plan(past, new, np.asarray(table)[:, :max_pages], max_pages, ring, cursor, page, num_tokens)
    for k in want:
        assert got[k] == [int(x) for x in want[k]], k
    np.testing.assert_array_equal(tab[:, :max_pages], wtab)
    np.testing.assert_array_equal(tab[:, max_pages:], np.asarray(table)[:, max_pages:])
    np.testing.assert_array_equal(rg, wrg)
    assert cur == wcur
    return want


def plan_case(seed, seqs, page, past_hi, new_hi, ended=0.1, short=None, spare=3, idle=0.1):
    rng = np.random.default_rng(seed)
    past = rng.integers(0, past_hi + 1, seqs)
    new = rng.integers(1, new_hi + 1, seqs)
    new[rng.random(seqs) < idle] = 0
    new[rng.random(seqs) < ended] = -1
    held = -(-past // page)
    need = int((-(-(past + np.maximum(new, 0)) // page) - held).sum())
    free = need + spare if short is None else max(0, need - short)
    pages = int(held.sum()) + free + 1
    ids = rng.permutation(pages)
    width = int(max(1, (-(-(past + np.maximum(new, 0)) // page)).max(initial=1)))
    table = np.full((max(1, seqs), width + 5), -9)
    at = 0
    for r in range(seqs):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    ring = np.full(pages, -3)
    head = int(rng.integers(pages))
    ring[(head + np.arange(free)) % pages] = ids[at:at + free]
    return past, new, table, width, ring, [head, free], page, int(np.maximum(new, 0).sum())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,page,past_hi,new_hi", [
    (1, 16, 0, 1), (1, 16, 15, 1), (1, 16, 5000, 3000), (2, 32, 100, 1), (63, 16, 40, 3), (64, 64, 700, 1), (65, 16, 33, 40),
    (255, 16, 100, 2), (256, 128, 900, 1), (257, 16, 50, 5), (700, 32, 300, 90), (4096, 16, 64, 1), (4095, 1024, 9000, 40)])
def test_plan_matches_the_definition(seqs, page, past_hi, new_hi, in_place):
    c = plan_case(seqs * 31 + page, seqs, page, past_hi, new_hi)
    check_plan(*c, in_place=in_place)


@pytest.mark.parametrize("short", [1, 3, 20, 10 ** 6])
@pytest.mark.parametrize("seqs", [1, 40, 600])
def test_plan_refuses_requests_when_pages_run_out(seqs, short):
    c = plan_case(seqs + short, seqs, 16, 100, 40, short=short)
    want = check_plan(*c)
    if short > 600 * 5:
        assert want["meta"][1] == 0 and want["meta"][3] > 0


@pytest.mark.parametrize("pad", [1, 64, 5000])
def test_plan_pads_the_tail(pad):
    *c, tokens = plan_case(9, 30, 16, 60, 9)
    check_plan(*c, tokens + pad)


def test_plan_without_requests_or_tokens():
    check_plan([], [], np.zeros((1, 3)), 3, [4, 5, 6], [1, 2], 16, 0)
    check_plan([], [], np.zeros((1, 3)), 3, [4, 5, 6], [1, 2], 16, 7)
    check_plan([5, 16], [0, -1], [[0, -1], [1, -1]], 2, [2, 3, -1, -1], [0, 2], 16, 0)


def test_plan_all_ended_fills_the_ring_over_its_end():
    seqs, page = 50, 16
    past = np.full(seqs, 40)
    table = np.arange(seqs * 3).reshape(seqs, 3)
    check_plan(past, np.full(seqs, -1), table, 3, np.full(seqs * 3 + 4, -1), [100, 4], page, 0)


def test_plan_wrong_words_stay_in_bounds():
    """Negative and overlong lengths, foreign page ids, a wrong cursor, too many tokens: counted, never followed."""
    big = 2 ** 31 - 1
    past = [-1, 5, 10, big, 17, 33, 40, 3]
    new = [1, -2, big, 1, 4, -1, 1, 13]
    table = np.full((8, 4), -1)
    table[4] = [10 ** 9, -5, -1, -1]
    table[5] = [3, 64, -7, -1]
    table[6] = [1, 2, big, -1]
    table[7] = [5, -1, -1, -1]
    ring = np.array([6, 7, -4, 99, 1, 2, 3, 4])
    got, tab, rg, cur = run_plan(past, new, table, 4, ring, [6, 5], 16, 12)
    # 1 + 1 + 1 + 1 for the lengths of requests 0..3; the tokens of request 2 (2^31 - 1) fill the batch
    assert got["query_start"] == [0, 0, 0, 12, 12, 12, 12, 12, 12]
    assert got["slots"] == [-1] * 12 and got["seq_lens"][:4] == [0, 0, 0, 0]
    assert got["seq_lens"][4:] == [21, 0, 41, 16]
    # request 5 gives back pages 3, 64 and -7 of a cache of 8: the two foreign ones as -1
    assert [rg[(6 + 5 + e) % 8] for e in range(3)] == [3, -1, -1]
    assert cur == [6, 8]
    for bad in ([-13, 5], [6, 10 ** 9], [-(2 ** 31), -1]):
        run_plan(past, new, table, 4, ring, bad, 16, 12)


def test_plan_on_another_stream_and_in_a_graph():
    """A captured step advances its own cursor; replays equal eager steps of the same requests."""
    past, new, table, width, ring, cursor, page, tokens = plan_case(3, 70, 16, 200, 3, ended=0, spare=10 ** 4)
    s = torch.cuda.Stream()
    eager = run_plan(past, new, table, width, ring, cursor, page, tokens, stream=s)
    plan = rx.PagePlan(0, 70, tokens)
    d = dict(past=ints(past), new=ints(new), ring=ints(ring), cursor=ints(cursor + [0, 0]), table=ints(table))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rx.page_plan(plan, d["past"], d["new"], tokens, d["ring"], d["cursor"], d["table"], page)
    cur = cursor
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        want, wtab, wrg, cur = KO.page_plan(past, new, table, width, ring, cur, page, tokens)
        assert plan.slots.tolist() == want["slots"] and d["cursor"].tolist() == cur + [0, 0]
        np.testing.assert_array_equal(d["table"].cpu().numpy()[:, :width], wtab[:, :width])
    assert eager[0]["slots"] == KO.page_plan(past, new, table, width, ring, cursor, page, tokens)[0]["slots"]


# =============================================================================== rotary append
def make_cache(cache, pages, page, heads, dim, order, seed, pad=0):
    """k, v [pages, page, heads, dim]; pad: elements left unused after every token's heads."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    two = []
    for _ in range(2):
        if order == "token":
            base = torch.randn(pages, page, heads * dim + pad, generator=g, device="cuda").to(DT[cache])
            two.append(base[:, :, :heads * dim].unflatten(2, (heads, dim)))
        else:
            base = torch.randn(pages, heads, page, dim + pad, generator=g, device="cuda").to(DT[cache])
            two.append(base[..., :dim].transpose(1, 2))
    return two


def rotary_case(seed, T, hq, kv, dim, rot, inter, cache, order, page=16, factor=1.0, amplitude=1.0, pos_hi=5000, pad=0):
    rng = np.random.default_rng(seed)
    act = act_of(cache)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    qkv = torch.randn(T, (hq + 2 * kv) * dim + pad, generator=g, device="cuda").to(act)[:, :(hq + 2 * kv) * dim]
    pages = -(-T // page) + 2
    k, v = make_cache(cache, pages, page, kv, dim, order, seed + 1, pad)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    positions = rng.integers(0, pos_hi, T)
    freqs = [f / factor for f in KO.frequencies(rot, 10000.0)]
    return qkv, k, v, slots, positions, freqs


def check_rotary(qkv, q_out, k, v, k0, v0, slots, positions, freqs, hq, kv, dim, inter, amplitude, scales, what):
    act, T, page = qkv.dtype, qkv.shape[0], k.shape[1]
    x = f64(qkv).reshape(T, hq + 2 * kv, dim)
    y, size = KO.rotate(x[:, :hq + kv], positions, freqs, inter, amplitude)
    rot = 2 * len(freqs)
    # fp32 cosine and sine (2^-22 of them, the fraction of a turn among it), two products, a sum; then one rounding
    slack = 2.0 ** -20 if act == BF else 2.0 ** -22
    half = HALF_STEP[act]
    got_q = f64(q_out).reshape(T, hq, dim)
    err = np.abs(got_q - y[:, :hq]) - half * np.abs(y[:, :hq])
    record_error(what, "q over step", float((err / size[:, :hq].clip(1e-30)).max(initial=0)), slack)
    assert (err <= slack * size[:, :hq]).all()
    assert (got_q[..., rot:] == x[:, :hq, rot:]).all()          # past rot_dim: unchanged
    want_k, want_v = f64(k0), f64(v0)
    got_k, got_v = f64(k), f64(v)
    ok = [t for t in range(T) if 0 <= slots[t] < k.shape[0] * page]
    at = np.array([slots[t] for t in ok], dtype=np.int64)
    pg, off = at // page, at % page
    yk, sk, xv = y[ok, hq:], size[ok, hq:], x[ok, hq + kv:]
    gk, gv = got_k[pg, off], got_v[pg, off]
    if k.dtype == E4M3:
        yk, sk, xv = yk / scales[0], sk / scales[0], xv / scales[1]
        for got, ref, size_ in ((gk, yk, sk), (gv, xv, np.abs(xv))):
            ref = np.clip(ref, -448, 448)
            # half a step: 2^-4 of the value, 2^-10 among the subnormals
            assert (np.abs(got - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10) + 2.0 ** -19 * size_).all()
            assert (np.isin(got, KO.e4m3_round(got))).all()
        # nearest even: all but values within the slack of a border
        assert (gv != KO.e4m3_round(xv)).mean() <= 1e-3 and (gk != KO.e4m3_round(yk)).mean() <= 1e-3
    else:
        assert (np.abs(gk - yk) <= half * np.abs(yk) + slack * sk).all()
        assert (gk[..., rot:] == x[ok, hq:hq + kv, rot:]).all() and (gv == xv).all()
    keep = np.ones(k.shape[:2], dtype=bool)
    keep[pg, off] = False
    np.testing.assert_array_equal(got_k[keep], want_k[keep])    # nothing else is written
    np.testing.assert_array_equal(got_v[keep], want_v[keep])


def run_rotary(T, hq, kv, dim, rot, inter, cache, order, seed=0, amplitude=1.0, factor=1.0, pos_hi=5000, page=16, pad=0,
               slots=None, positions=None, in_place=False, scales=(0.5, 2.0)):
    qkv, k, v, sl, pos, freqs = rotary_case(seed, T, hq, kv, dim, rot, inter, cache, order, page, factor, amplitude, pos_hi, pad)
    sl, pos = sl if slots is None else np.asarray(slots), pos if positions is None else np.asarray(positions)
    scales = scales if cache == "fp8" else (1.0, 1.0)
    k0, v0, x0 = k.clone(), v.clone(), qkv.clone()
    q = qkv[:, :hq * dim] if in_place else torch.full((T, hq * dim + pad), 7.0, dtype=qkv.dtype, device="cuda")[:, :hq * dim]
    r = rx.Rotary(0, rot, freqs, interleaved=inter, amplitude=amplitude)
    rx.rotary_append(r, qkv, hq, ints(pos), ints(sl), q, rx.KVCache(k, v, *scales))
    torch.cuda.synchronize()
    check_rotary(x0, q, k, v, k0, v0, sl, pos, freqs, hq, kv, dim, inter, amplitude, scales,
                 f"T={T} {hq}/{kv}x{dim} rot={rot} {cache}")
    if not in_place:
        assert torch.equal(qkv, x0)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(16, 2), (16, 16), (64, 64), (80, 20), (80, 40), (96, 72), (128, 64), (128, 128), (192, 66),
                                     (256, 256), (128, 24), (64, 6)])
def test_rotary_layouts(dim, rot, inter, cache):
    run_rotary(13, 6, 2, dim, rot, inter, cache, "token", seed=dim + rot)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("T,hq,kv", [(1, 1, 1), (1, 32, 8), (2, 8, 8), (7, 5, 1), (64, 32, 8), (333, 12, 4), (1025, 4, 2)])
def test_rotary_sizes(T, hq, kv, cache):
    run_rotary(T, hq, kv, 128, 128, False, cache, "head" if T % 2 else "token", seed=T, page=64 if T > 7 else 16)


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
def test_rotary_strides(cache, order):
    """Rows and cache cells with unused elements between them."""
    run_rotary(21, 8, 4, 64, 32, False, cache, order, seed=5, pad=48, page=32)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_in_place(cache, inter):
    run_rotary(40, 8, 2, 128, 96, inter, cache, "token", seed=8, in_place=True)
    run_rotary(3, 8, 2, 80, 20, inter, cache, "token", seed=9, in_place=True)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_rotary_far_positions(cache):
    pos = [0, 1, 2 ** 20, 2 ** 24 + 1, 2 ** 30, 2 ** 31 - 1, -1, -(2 ** 31)]
    run_rotary(8, 4, 2, 64, 64, False, cache, "token", seed=2, positions=pos, amplitude=1.25)


def test_rotary_slots_outside_the_cache_store_nothing():
    for bad in ([-1] * 9, [-1, 3, 48, 2 ** 31 - 1, -(2 ** 31), 47, 10 ** 6, 0, 49]):
        run_rotary(9, 4, 2, 64, 64, False, "bf16", "token", seed=4, slots=bad)


def test_rotary_no_tokens():
    run_rotary(0, 4, 2, 64, 64, False, "bf16", "token")


@pytest.mark.parametrize("cache", ["bf16", "fp8", "f32"])
def test_rotary_infinities_and_nan_stay_in_their_pair(cache):
    T, hq, kv, dim, rot = 3, 2, 1, 64, 32
    qkv, k, v, slots, pos, freqs = rotary_case(1, T, hq, kv, dim, rot, False, cache, "token")
    qkv[1, 5], qkv[1, dim + 40], qkv[2, 3 * dim + 7], qkv[0, 2 * dim + 50] = float("nan"), float("inf"), float("nan"), -float("inf")
    q = torch.zeros(T, hq * dim, dtype=qkv.dtype, device="cuda")
    rx.rotary_append(rx.Rotary(0, rot, freqs), qkv, hq, ints(pos), ints(slots), q, rx.KVCache(k, v))
    bad = torch.nonzero(~torch.isfinite(q.float())).tolist()
    assert bad == [[1, 5], [1, 5 + rot // 2], [1, dim + 40]]
    gv = v[slots[2] // 16, slots[2] % 16, 0].float()
    assert torch.isnan(gv[7]) and torch.isfinite(gv).sum() == dim - 1
    gk = k[slots[0] // 16, slots[0] % 16, 0].float()
    assert gk[50] == (-448.0 if cache == "fp8" else -float("inf"))


# =============================================================================== attention
def attend_case(seed, lens, news, hq, kv, dim, cache, order, page=16, pad=0, spread=1.0):
    rng = np.random.default_rng(seed)
    act = act_of(cache)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    k, v = make_cache(cache, pages, page, kv, dim, order, seed + 1, pad)
    ids = rng.permutation(pages)
    table = np.full((len(lens), max([1] + need) + 1), -1)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    T = sum(news)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q = (torch.randn(T, hq * dim + pad, generator=g, device="cuda") * spread).to(act)[:, :hq * dim]
    return q, k, v, table, np.concatenate([[0], np.cumsum(news)]).astype(int)


def poison_unseen(k, v, table, lens, page, value):
    """`value` at every cached place that no sequence holds."""
    held = torch.zeros(k.shape[:2], dtype=torch.bool)
    for r, n in enumerate(lens):
        for j in range(n):
            if 0 <= table[r][j // page] < k.shape[0]:
                held[table[r][j // page], j % page] = True
    for x in (k, v):
        bits = x.view(torch.uint8) if x.dtype == E4M3 else x
        fill = 0x7F if x.dtype == E4M3 else value
        bits[~held.cuda()] = fill


def check_attend(q, k, v, table, lens, starts, page, hq, kv, dim, out, lse, scale, window, scales, what, rows=None):
    T = q.shape[0]
    Q, K, V = f64(q).reshape(T, hq, dim), f64(k) * scales[0], f64(v) * scales[1]
    ref, rl, mass, smax = KO.attend(Q, np.nan_to_num(K), np.nan_to_num(V), table, lens, starts, page, scale, window)
    L = max([1] + list(lens))
    act = q.dtype
    # scores: products and sums of dim terms in fp32, the scale, and the exponential's argument in base 2; then the
    # exponential (2^-20), for bf16 the weights in two bf16 parts (2^-16), the sums of up to L terms, one rounding
    ds = smax[..., None] * (dim + 16) * 2.0 ** -24
    rel = 2 * ds + (2.0 ** -15 if act == BF else 2.0 ** -19) + (L + 64) * 2.0 ** -24
    tol = HALF_STEP[act] * np.abs(ref) + mass * rel * 1.01
    got, gl = f64(out).reshape(T, hq, dim), f64(lse)
    rows = slice(None) if rows is None else rows
    err = np.abs(got - ref)[rows]
    record_error(what, "of tolerance", float((err / tol[rows].clip(1e-30)).max(initial=0)), 1.0)
    assert np.isfinite(got[rows]).all()
    assert (err <= tol[rows]).all()
    empty = np.isneginf(rl)
    assert (np.isneginf(gl) == empty)[rows].all() and (got[empty] == 0)[...].all()
    rl0, gl0 = np.where(empty, 0, rl), np.where(empty, 0, gl)
    # ln of the sum: the scores' error, the sum's relative error, its own rounding
    tl = ds[..., 0] + (L + 64) * 2.0 ** -24 + 2.0 ** -20 + np.abs(rl0) * 2.0 ** -22
    assert (np.abs(gl0 - rl0) <= tl)[rows].all()


def run_attend(lens, news, hq, kv, dim, cache, order="token", page=16, window=0, seed=0, pad=0, spread=1.0, poison=float("nan"),
               scale=None, table_edit=None):
    q, k, v, table, starts = attend_case(seed, lens, news, hq, kv, dim, cache, order, page, pad, spread)
    if poison is not None:
        poison_unseen(k, v, table, lens, page, poison)
    if table_edit is not None:
        table_edit(table)
    scales = (0.75, 1.5) if cache == "fp8" else (1.0, 1.0)
    scale = dim ** -0.5 if scale is None else scale
    T = q.shape[0]
    out = torch.full((T, hq * dim + pad), 7.0, dtype=q.dtype, device="cuda")[:, :hq * dim]
    lse = torch.full((T, hq), 7.0, dtype=F32, device="cuda")
    att = rx.Attention(0, max(1, len(lens)), max(1, T), hq, kv, dim)
    args = (att, q, rx.KVCache(k, v, *scales), ints(table), ints(lens), ints(starts), out)
    rx.paged_attention(*args, scale=scale, window=window, lse=lse)
    torch.cuda.synchronize()
    check_attend(q, k, v, table, lens, starts, page, hq, kv, dim, out, lse, scale, window, scales,
                 f"{len(lens)} seqs to {max(lens)} {hq}/{kv}x{dim} {cache} window={window}")
    first, first_lse = out.clone(), lse.clone()
    out.fill_(3.0)
    rx.paged_attention(*args, scale=scale, window=window)
    torch.cuda.synchronize()
    assert torch.equal(out, first)                      # the same bits again, with or without lse
    return first, first_lse


CACHES = ["bf16", "fp8", "f32"]


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700])
def test_attention_lengths(n, cache):
    run_attend([n], [1], 8, 2, 64, cache, seed=n)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 208, 256])
def test_attention_head_dims(dim, cache):
    run_attend([70, 3, 200], [1, 1, 1], 6, 2, dim, cache, order="head" if dim % 32 else "token", seed=dim)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("hq,kv", [(1, 1), (4, 4), (3, 1), (7, 1), (8, 1), (15, 1), (16, 1), (17, 1), (32, 1), (40, 2), (33, 1), (71, 1)])
def test_attention_head_groups(hq, kv, cache):
    run_attend([90, 41], [1, 1], hq, kv, 64, cache, seed=hq)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("news", [[2, 2, 2], [4, 1, 7], [1, 33, 5], [3, 16, 0], [0, 50, 1]])
@pytest.mark.parametrize("window", [0, 20])
def test_attention_several_new_tokens(news, window, cache):
    run_attend([77, 50, 130], news, 8, 2, 64, cache, seed=sum(news), window=window)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("window", [1, 5, 16, 31, 32, 100, 1000, 2 ** 31 - 1])
def test_attention_windows(window, cache):
    run_attend([1, 40, 333, 900], [1, 1, 1, 2], 4, 2, 128, cache, seed=window % 97, window=window)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf"), None])
@pytest.mark.parametrize("cache", CACHES)
def test_attention_ignores_what_it_does_not_see(cache, poison):
    run_attend([5, 37, 64, 301], [1, 3, 1, 2], 4, 2, 64, cache, seed=3, poison=poison, window=0)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_unseen_places_between_the_rows_of_a_tile(cache, bad):
    """A key that only later tokens of the block see (and one that has left the window of later ones) holds NaN or
    infinities: the rows that do not see it are untouched."""
    lens, news, window = [60], [5], 40
    q, k, v, table, starts = attend_case(6, lens, news, 4, 2, 64, cache, "token")
    clean_k, clean_v = k.clone(), v.clone()
    for j in (57, 59, 17):       # tokens 0..4 stand at 55..59; 17 is seen up to position 56
        for x in (k, v):
            x[table[0][j // 16], j % 16] = bad
    att = rx.Attention(0, 1, 5, 4, 2, 64)
    out, lse = torch.zeros_like(q), torch.zeros(5, 4, device="cuda")
    rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), out, window=window, lse=lse)
    want = torch.zeros_like(q)
    rx.paged_attention(att, q, rx.KVCache(clean_k, clean_v), ints(table), ints(lens), ints(starts), want, window=window)
    torch.cuda.synchronize()
    for i in range(5):
        sees = any(55 + i - window < j <= 55 + i for j in (57, 59, 17))
        assert torch.isfinite(out[i].float()).all().item() != sees, i
        if not sees:
            assert torch.equal(out[i], want[i]) or (out[i].float() - want[i].float()).abs().max() <= 2.0 ** -7 * want[i].float().abs().max()


@pytest.mark.parametrize("cache", CACHES)
def test_attention_rows_that_see_nothing(cache):
    out, lse = run_attend([0, 10, 0, 3], [1, 1, 2, 5], 4, 2, 64, cache, seed=1)   # sequence 3: two tokens stand before 0
    assert not out[0].any() and torch.isneginf(lse[0]).all() and not out[4:6].any()


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_wrong_pages_are_left_out(cache, dim):
    def edit(table):
        table[0][1], table[1][0], table[1][2], table[2][:] = -1, 10 ** 9, -(2 ** 31), -7
    run_attend([60, 55, 40, 100], [1, 2, 1, 1], 4, 2, dim, cache, seed=2, poison=None, table_edit=edit)


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("cache", CACHES)
def test_attention_strides(cache, order):
    run_attend([100, 7], [1, 2], 8, 4, 80, cache, order=order, page=32, pad=48, seed=4)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
def test_attention_pages(page, cache):
    run_attend([page - 1, page, page + 1, 3 * page + 5], [1, 1, 2, 1], 4, 1, 64, cache, page=page, seed=page)


@pytest.mark.parametrize("cache", CACHES)
def test_attention_large_scores(cache):
    """Scores of some hundreds: the running maximum moves far and often."""
    run_attend([300, 64], [1, 2], 4, 2, 128, cache, seed=7, spread=40.0)
    run_attend([300, 64], [1, 2], 4, 2, 128, cache, seed=8, scale=-0.3)
    run_attend([300, 64], [1, 2], 4, 2, 128, cache, seed=8, scale=0.0)


@pytest.mark.parametrize("seqs", [5, 64, 257, 600])
def test_attention_many_sequences(seqs):
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 90, seqs)
    lens[0] = 700
    news = rng.integers(0, 3, seqs)
    news[0] = 1
    run_attend(lens.tolist(), np.minimum(news, np.maximum(lens, 1)).tolist(), 4, 2, 64, "bf16", seed=seqs)


@pytest.mark.parametrize("cache", CACHES)
def test_attention_long_sequence_beside_short_ones(cache):
    run_attend([20001, 3, 900], [1, 1, 2], 4, 1, 64, cache, page=64, seed=11)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_attention_offsets_past_32_bits(cache):
    """Pages 2^27 elements apart: byte and element offsets beyond 2^31 and 2^32."""
    dim, kv, page, pages = 64, 2, 16, 40
    stride = 1 << 27
    ks = []
    for _ in range(2):
        base = torch.empty((pages - 1) * stride + page * kv * dim, dtype=DT[cache], device="cuda")
        ks.append(base.as_strided((pages, page, kv, dim), (stride, kv * dim, dim, 1)))
    q, k, v, table, starts = attend_case(3, [600], [2], 4, kv, dim, cache, "token")
    for x, src in zip(ks, (k, v)):
        (x.view(torch.uint8) if cache == "fp8" else x).copy_((src.view(torch.uint8) if cache == "fp8" else src))
    out, want, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(2, 4, device="cuda")
    att = rx.Attention(0, 1, 2, 4, kv, dim)
    rx.paged_attention(att, q, rx.KVCache(*ks), ints(table), ints([600]), ints(starts), out, lse=lse)
    rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints([600]), ints(starts), want)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and out.any()
    # and the append into the same cache
    T = 5
    qkv = torch.randn(T, (4 + 2 * kv) * dim, device="cuda").to(BF)
    slots, pos = ints([39 * 16 + 3, 17 * 16, 35 * 16 + 15, 1, 38 * 16]), ints([7, 8, 9, 10, 11])
    r = rx.Rotary(0, dim, KO.frequencies(dim, 10000.0))
    qo = torch.zeros(T, 4 * dim, dtype=BF, device="cuda")
    rx.rotary_append(r, qkv, 4, pos, slots, qo, rx.KVCache(*ks))
    rx.rotary_append(r, qkv, 4, pos, slots, qo, rx.KVCache(k, v))
    torch.cuda.synchronize()
    for x, src in zip(ks, (k, v)):
        a, b = ((y.view(torch.uint8) if cache == "fp8" else y) for y in (x, src))
        assert torch.equal(a.contiguous(), b.contiguous())


def test_attention_wrong_starts_and_lengths_stay_in_bounds():
    """Rows that belong to no sequence are left alone, wrong words are taken at their bounds."""
    q, k, v, table, _ = attend_case(5, [50, 60], [3, 4], 4, 2, 64, "bf16", "token")
    att = rx.Attention(0, 2, 7, 4, 2, 64)
    out = torch.full_like(q, 7.0)
    rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints([50, 60]), ints([0, 2, 5]), out)
    torch.cuda.synchronize()
    assert (out[5:] == 7).all() and (out[:5] != 7).any(1).all()
    for starts, lens in (([5, 2, 9], [50, 60]), ([-4, 3, 2 ** 31 - 1], [2 ** 31 - 1, -5]), ([0, 7, 0], [50, 60]),
                         ([2 ** 31 - 1, -(2 ** 31), 4], [10 ** 6, 60])):
        rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), out)
        torch.cuda.synchronize()
    # the object works on after them
    good = torch.zeros_like(q)
    rx.paged_attention(att, q, rx.KVCache(k, v), ints(table), ints([50, 60]), ints([0, 3, 7]), good)
    ref, *_ = KO.attend(f64(q).reshape(7, 4, 64), f64(k), f64(v), table, [50, 60], [0, 3, 7], 16, 0.125)
    assert np.abs(f64(good).reshape(7, 4, 64) - ref).max() < 0.03


def test_attention_object_for_steps_of_different_sizes_streams_and_graphs():
    """One object, its workspace reused by steps of other sizes, on another stream, in a graph between eager calls."""
    dim, hq, kv = 128, 8, 2
    cases = [attend_case(20 + i, lens, news, hq, kv, dim, "bf16", "token") + (lens,) for i, (lens, news) in enumerate(
        [([5000], [1]), ([30, 700, 1200], [1, 1, 1]), ([64] * 40, [1] * 40), ([3000, 10], [4, 1])])]
    want = []
    for q, k, v, table, starts, lens in cases:
        one = rx.Attention(0, len(lens), q.shape[0], hq, kv, dim)
        o = torch.zeros_like(q)
        rx.paged_attention(one, q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), o)
        torch.cuda.synchronize()
        want.append(o)
    att = rx.Attention(0, 64, 64, hq, kv, dim)
    args = [(q, rx.KVCache(k, v), ints(table), ints(lens), ints(starts), torch.zeros_like(q)) for q, k, v, table, starts, lens in cases]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for rep in range(2):
        for a, w in zip(args, want):
            a[-1].fill_(9.0)
            s.wait_stream(torch.cuda.current_stream())
            rx.paged_attention(att, *a, stream=s)
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize()
            # the split depends on the step, not on the object: bitwise equal
            assert torch.equal(a[-1], w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rx.paged_attention(att, *args[0])
        rx.paged_attention(att, *args[3])
    for rep in range(4):
        for a in args:
            a[-1].fill_(rep + 1.0)
        rx.paged_attention(att, *args[1])
        g.replay()
        rx.paged_attention(att, *args[2])
        torch.cuda.synchronize()
        for a, w in zip(args, want):
            assert torch.equal(a[-1], w)


def test_timing_names_the_new_kernels():
    rx.lora_timing_enable(True)
    try:
        rx.lora_timing_report()
        run_plan([5], [1], [[0, 1]], 2, [2, 3, 1], [0, 2], 16, 1)
        run_rotary(2, 4, 2, 64, 64, False, "bf16", "token")
        run_attend([20], [1], 4, 2, 64, "bf16")
        rep = rx.lora_timing_report()
    finally:
        rx.lora_timing_enable(False)
    for name in ("page_plan", "rotary_append", "attention"):
        assert rep[name][1] >= 1 and rep[name][0] > 0
