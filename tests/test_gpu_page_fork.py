"""Page forks and page copies on the GPU against their definitions (oracle/beam_oracle.py)."""
import numpy as np
import pytest
import torch

import oracle.beam_oracle as BO
import rank_adapter_gemm_build_amd as rx

pytestmark = pytest.mark.gpu

I32, BF, F32, E4M3 = torch.int32, torch.bfloat16, torch.float32, torch.float8_e4m3fn
DT = {"bf16": BF, "f32": F32, "fp8": E4M3}
OUT = ("copy_src", "copy_dst", "copy_tokens", "meta")


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


class State:
    """A block table whose rows share pages, with the ring and the counts, kept beside its definition's."""

    def __init__(self, seed, rows, page, len_hi, free, spare_columns=3, elsewhere=2):
        rng = np.random.default_rng(seed)
        self.page, self.rows = page, rows
        self.lens = rng.integers(0, len_hi + 1, rows)
        self.width = max(1, -(-len_hi // page))
        table, shares = np.full((rows, self.width + spare_columns), -9), []
        at = 0
        for r in range(rows):
            donor = int(rng.integers(0, r)) if r and rng.random() < 0.7 else -1
            both = min(self.lens[r], self.lens[donor]) // page if donor >= 0 else 0
            both = int(rng.integers(0, both + 1))
            for c in range(-(-self.lens[r] // page)):
                if c < both:
                    table[r, c] = table[donor, c]
                    shares[table[r, c]] += 1
                else:
                    table[r, c] = at
                    shares.append(0)
                    at += 1
        N = at + free + elsewhere
        ids = rng.permutation(N)
        self.table = np.where(table >= 0, ids[np.clip(table, 0, None)], table)
        self.shares = np.zeros(N, dtype=np.int64)
        self.shares[ids[:at]] = shares
        self.ring = np.full(N, -3)
        head = int(rng.integers(N))
        self.ring[(head + np.arange(free)) % N] = ids[at:at + free]
        self.cursor, self.N, self.rng = [head, free], N, rng

    def random_parents(self, group=0, gone=0.1):
        base = np.arange(self.rows) // group * group if group else np.zeros(self.rows, dtype=np.int64)
        size = np.minimum(group, self.rows - base) if group else np.full(self.rows, self.rows)
        p = base + (self.rng.random(self.rows) * size).astype(np.int64)
        p[self.rng.random(self.rows) < gone] = -1
        return p

    def device(self):
        """The call's vectors between margins."""
        self.margins = {}

        def vec(values, name):
            v = torch.full((len(values) + 32,), -55, dtype=I32, device="cuda")
            v[16:-16] = ints(values)
            self.margins[name] = v
            return v[16:-16]
        self.d = {"lens": vec(self.lens, "lens"), "free_pages": vec(self.ring, "ring"), "cursor": vec(self.cursor + [0, 0], "cursor"),
                  "shares": vec(self.shares, "shares"), "block_table": ints(self.table)}
        self.plan = rx.ForkPlan(0, min(self.rows + 3, rx.LORA_MAX_SEQS), self.N)
        for k in OUT:
            getattr(self.plan, k).fill_(-77)
        return self

    def fork(self, parents, stream=None):
        d = self.d
        rx.page_fork(self.plan, ints(parents), d["lens"], d["free_pages"], d["cursor"], d["shares"], d["block_table"][:, :self.width],
                     self.page, stream=stream)

    def check(self, parents, what=""):
        torch.cuda.synchronize()
        want, lens, table, ring, cursor, shares = BO.page_fork(parents, self.lens, self.table[:, :self.width], self.width, self.ring,
                                                               self.cursor, self.shares, self.page)
        got = {k: getattr(self.plan, k).cpu().numpy() for k in OUT}
        for k in OUT:
            assert got[k][:len(want[k])].tolist() == want[k], (what, k)
            if k != "meta":
                assert (got[k][self.rows:] == -77).all(), (what, k)
        self.table[:, :self.width] = table
        self.lens, self.ring, self.cursor, self.shares = np.array(lens), np.array(ring), cursor, np.array(shares)
        self.same(what)
        return want

    def same(self, what=""):
        d = self.d
        assert d["lens"].tolist() == self.lens.tolist(), what
        np.testing.assert_array_equal(d["block_table"].cpu().numpy(), self.table, err_msg=what)
        assert d["free_pages"].tolist() == self.ring.tolist(), what
        assert d["cursor"].tolist() == list(self.cursor) + [0, 0], what
        assert d["shares"].tolist() == self.shares.tolist(), what
        assert not self.plan._scratch.any(), what
        for k, v in self.margins.items():
            assert (v[:16] == -55).all() and (v[-16:] == -55).all(), (what, k)

    def holders(self):
        """Every page's holders from the table itself."""
        n = np.zeros(self.N, dtype=np.int64)
        for r in range(self.rows):
            n[self.table[r, :-(-self.lens[r] // self.page)]] += 1
        return n


@pytest.mark.parametrize("rows,page,len_hi", [(1, 16, 1), (1, 16, 5000), (2, 16, 15), (4, 16, 777), (5, 32, 64), (63, 16, 400), (64, 1024, 5000),
                                              (65, 16, 100), (255, 64, 900), (257, 16, 70), (1000, 16, 300), (1024, 128, 3000), (4096, 16, 40)])
def test_fork_matches_the_definition(rows, page, len_hi):
    s = State(rows + page, rows, page, len_hi, free=2 * rows + 5).device()
    for step, group in enumerate((0, 4, 8, 1)):
        parents = s.random_parents(group)
        s.fork(parents)
        s.check(parents, f"step {step}")
    # counts of holders and ring account for every page
    n = s.holders()
    head, free = s.cursor
    ring = [int(s.ring[(head + i) % s.N]) for i in range(free)]
    assert len(set(ring)) == free and not n[ring].any()
    assert (s.shares == np.maximum(n - 1, 0)).all()


@pytest.mark.parametrize("rows", [1, 3, 8, 300])
def test_rows_that_stay_change_nothing_and_rows_that_end_free_their_pages(rows):
    s = State(rows, rows, 16, 200, free=4).device()
    before = s.table.copy(), s.shares.copy()
    s.fork(np.arange(rows))
    want = s.check(np.arange(rows))
    assert (s.table == before[0]).all() and (s.shares == before[1]).all() and want["meta"][:4] == [0, 0, 0, 0]
    s.fork([-1] * rows)
    s.check([-1] * rows)
    assert s.cursor[1] == s.N - 2 and not s.lens.any() and not s.shares.any()
    s.fork([-1] * rows)       # and nothing twice
    assert s.check([-1] * rows)["meta"][1] == 0


@pytest.mark.parametrize("free", [0, 1, 5])
def test_children_past_the_free_pages_are_refused(free):
    for seed in range(4):
        s = State(seed, 40, 16, 100, free=free).device()
        parents = s.random_parents(8, gone=0)
        s.fork(parents)
        want = s.check(parents)
        assert want["meta"][0] <= free
        if want["meta"][2]:
            assert want["meta"][0] == free


def test_all_children_of_one_row():
    for length in (0, 1, 16, 31, 1600):
        s = State(3, 100, 16, 1700, free=200).device()
        s.lens[7] = min(length, s.lens[7]) if length else 0
        s = s.device()
        s.fork([7] * 100)
        s.check([7] * 100)


def test_wrong_words_stay_in_bounds():
    """Parents, lengths, page ids, counts and cursors out of range: counted, never followed."""
    big = 2 ** 31 - 1
    s = State(9, 12, 16, 60, free=6)
    s.lens[[1, 2]] = [-5, big]
    s.table[4, 0], s.table[5, 1], s.table[6, 0] = 10 ** 9, -4, s.N
    s.lens[[4, 5, 6]] = [40, 41, 17]
    s.ring[(s.cursor[0] + 1) % s.N] = 10 ** 8
    s.device()
    parents = np.array([4, 4, 5, 5, -2, 12, big, 6, 1, 2, 3, 3])
    s.fork(parents)
    s.check(parents)
    for cursor in ([-13, 5], [3, 10 ** 9], [-(2 ** 31), -1]):
        s.cursor = cursor
        s.device()
        parents = s.random_parents()
        s.fork(parents)
        torch.cuda.synchronize()
        assert 0 <= s.d["cursor"][0] < s.N and 0 <= s.d["cursor"][1] <= s.N
    s.cursor = [0, 0]
    s.shares[:] = [-(2 ** 31), big, -1, 0] * (s.N // 4) + [0] * (s.N % 4)
    s.device()
    s.fork(s.random_parents())
    torch.cuda.synchronize()


def test_the_same_page_twice_in_wrong_tables_is_freed_once():
    s = State(2, 6, 16, 60, free=3)
    s.lens[:] = 64
    s.width = 4
    s.table[:, :4] = s.table[0, 0] if s.table[0, 0] >= 0 else 0
    s.shares[:] = 0
    s.device()
    s.fork([-1] * 6)
    s.check([-1] * 6)


@pytest.mark.parametrize("rows", [4, 1024])
def test_a_captured_fork_replays(rows):
    s = State(rows, rows, 16, 200, free=2 * rows).device()
    parents = ints(np.zeros(rows))
    d = s.d

    def call():
        rx.page_fork(s.plan, parents, d["lens"], d["free_pages"], d["cursor"], d["shares"], d["block_table"][:, :s.width], s.page)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        p = s.random_parents(4)
        parents.copy_(ints(p))
        g.replay()
        s.check(p, "replayed")


def test_fork_on_another_stream():
    s = State(5, 50, 32, 300, free=100).device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    parents = s.random_parents(5)
    s.fork(parents, stream=side)
    s.check(parents)


# =============================================================================== page copy
def cells(kind, layers, pages, page, heads, dim, order, pad, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if order == "token":
        x = torch.randn(layers, pages, page, heads * dim + pad, generator=g, device="cuda").to(DT[kind])
        return x, x[..., :heads * dim].unflatten(3, (heads, dim))
    x = torch.randn(layers, pages, heads, page, dim + pad, generator=g, device="cuda").to(DT[kind])
    return x, x[..., :dim].transpose(2, 3)


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("order,pad", [("token", 0), ("head", 0), ("token", 32), ("head", 16)])
@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("layers,pairs,page,heads,dim", [(1, 1, 16, 1, 16), (3, 7, 16, 2, 80), (2, 33, 64, 8, 128), (5, 4, 32, 3, 256), (128, 2, 16, 1, 64),
                                                         (1, 600, 16, 5, 48), (1, 3, 1024, 2, 32)])
def test_copy_matches_the_definition(layers, pairs, page, heads, dim, kind, order, pad):
    rng = np.random.default_rng(pairs)
    pages = 2 * pairs + 3
    (kb, k), (vb, v) = (cells(kind, layers, pages, page, heads, dim, order, pad, s) for s in (1, 2))
    ids = rng.permutation(pages)
    src, dst = ids[rng.integers(0, pairs, pairs)], ids[pairs:2 * pairs]
    tokens = rng.integers(0, page + 1, pairs)
    caches = [rx.KVCache(a, b) for a, b in zip(k, v)]
    arg = caches[0] if layers == 1 else rx.KVLayers(caches)
    for t in (tokens, None):
        before = [raw(x) for x in (kb, vb)]
        wants = []
        for x in (k, v):
            y = raw(x).reshape(layers, pages, page, -1)
            wants.append(np.stack([BO.page_copy(y[i], src, dst, t, page) for i in range(layers)]))
        rx.page_copy(arg, ints(src), ints(dst), None if t is None else ints(t))
        torch.cuda.synchronize()
        for x, want in zip((k, v), wants):
            assert (raw(x).reshape(want.shape) == want).all()
        if pad:                                           # what lies between the rows
            width = (heads * dim if order == "token" else dim) * k.element_size()
            for x, b in zip((kb, vb), before):
                rows = raw(x).reshape(-1, width + pad * k.element_size())
                assert (rows[:, width:] == b.reshape(rows.shape)[:, width:]).all()


def test_pairs_that_copy_nothing():
    _, k = cells("bf16", 1, 6, 16, 2, 32, "token", 0, 1)
    _, v = cells("bf16", 1, 6, 16, 2, 32, "token", 0, 2)
    cache = rx.KVCache(k[0], v[0])
    before = raw(k), raw(v)
    rx.page_copy(cache, ints([-1, 0, 6, 2, 10 ** 9, 3]), ints([1, -1, 2, 2, 4, -2 ** 31]), ints([16, 16, 16, 16, 16, 16]))
    rx.page_copy(cache, ints([0, 1]), ints([2, 3]), ints([0, -4]))
    rx.page_copy(cache, ints([]), ints([]))
    torch.cuda.synchronize()
    assert (raw(k) == before[0]).all() and (raw(v) == before[1]).all()
    rx.page_copy(cache, ints([0]), ints([2]), ints([10 ** 6]))     # taken as the page's size
    torch.cuda.synchronize()
    assert torch.equal(k[0, 2], k[0, 0]) and torch.equal(v[0, 2], v[0, 0])


def test_a_copy_far_into_a_large_cache():
    """Offsets past 32 bits."""
    pages = 2 ** 20 + 9                                   # of 4 KB: 4.3 GB of keys
    k = torch.zeros(pages, 16, 1, 128, dtype=BF, device="cuda")
    v = torch.zeros(pages, 16, 1, 128, dtype=BF, device="cuda")
    k[pages - 2].normal_()
    v[pages - 2].normal_()
    rx.page_copy(rx.KVCache(k, v), ints([pages - 2, pages - 2]), ints([pages - 1, 3]))
    torch.cuda.synchronize()
    for x in (k, v):
        assert torch.equal(x[pages - 1], x[pages - 2]) and torch.equal(x[3], x[pages - 2]) and not x[4].any()
