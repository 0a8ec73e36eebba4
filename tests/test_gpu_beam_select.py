"""Beam selection on the GPU against its 64-bit definition (oracle/beam_oracle.py)."""
import math

import numpy as np
import pytest
import torch

import oracle.beam_oracle as BO
import rank_adapter_gemm_build_amd as rx
from lora_cases import record_error

pytestmark = pytest.mark.gpu

I32, BF, F32 = torch.int32, torch.bfloat16, torch.float32
LOG_SUM = 2.0 ** -18      # the contract's bound on a log sum
HALF_STEP = 2.0 ** -24    # rounding of a score to float32, relative


def ints(x):
    return torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")


def floats(x):
    return torch.tensor(np.asarray(x, dtype=np.float32), device="cuda")


def make(seed, requests, beams, vocab, dtype=BF, pad=0, sigma=3.0, offset=0):
    """logits [rows, vocab] inside a wider matrix of NaN, `offset` values after its start."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = requests * beams
    flat = torch.full((rows * (vocab + pad) + offset + 64,), math.nan, dtype=dtype, device="cuda")
    x = flat[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    x.copy_(torch.randn((rows, vocab), generator=g, device="cuda") * sigma)
    scores = -np.random.default_rng(seed).random(rows).astype(np.float32) * 8
    return x, scores


class Out:
    def __init__(self, n, margin=16):
        self.n, self.margin = n, margin
        self.v = {k: torch.full((n + 2 * margin,), -77, dtype=F32 if k == "scores" else I32, device="cuda")
                  for k in ("parents", "tokens", "scores", "ended")}

    def __getitem__(self, k):
        return self.v[k][self.margin:self.margin + self.n]

    def check_margins(self):
        for k, v in self.v.items():
            assert (v[:self.margin] == -77).all() and (v[self.margin + self.n:] == -77).all(), k


def run(x, scores, beams, best, ended=None, end_token=-1, weights=None, obj=None, stream=None):
    rows, vocab = x.shape
    obj = obj or rx.Beams(0, max(1, rows // beams), beams, vocab, best)
    out = Out(rows // beams * best)
    rx.beam_select(obj, x, floats(scores), out["parents"], out["tokens"], out["scores"], ended=None if ended is None else ints(ended),
                   end_token=end_token, ended_out=out["ended"], weights=None if weights is None else floats(weights), stream=stream)
    torch.cuda.synchronize()
    out.check_margins()
    return {k: out[k].cpu().numpy() for k in out.v}


def compare(got, x, scores, beams, best, ended=None, end_token=-1, weights=None, what=""):
    """Parents and tokens equal the definition's; candidates of two rows may change places where their ranks differ by
    less than the log sums' bound."""
    logits = x.double().cpu().numpy()
    want = BO.select(logits, scores, beams, best, ended, end_token, weights)
    lse = BO.log_sums(logits)
    worst = 0.0
    for r, found in enumerate(want):
        at = slice(r * best, r * best + best)
        par, tok, sc, end = got["parents"][at], got["tokens"][at], got["scores"][at], got["ended"][at]
        n = len(found)
        assert (par[n:] == -1).all() and (tok[n:] == -1).all() and (sc[n:] == -np.inf).all() and (end[n:] == 0).all(), what
        assert len(set(zip(par[:n].tolist(), tok[:n].tolist()))) == n, what
        for c, (rank, row, token, score, done) in enumerate(found):
            w = 1.0 if weights is None else float(weights[row])
            if (par[c], tok[c]) != (row, token):
                p, t = int(par[c]), int(tok[c])
                assert p != row and r * beams <= p < (r + 1) * beams, (what, r, c, (p, t), (row, token))
                other = float(scores[p]) if ended is not None and ended[p] else float(scores[p]) + (logits[p, t] - lse[p])
                v = 1.0 if weights is None else float(weights[p])
                assert abs(other * v - rank) <= 2 * LOG_SUM * max(w, v), (what, r, c)
                score, done = other, int((ended is not None and ended[p]) or t == end_token)
            assert end[c] == done, what
            worst = max(worst, abs(float(sc[c]) - score) / (LOG_SUM + HALF_STEP * abs(score)))
    record_error(f"beam selection {what}: scores against their bound", "rel", worst, 1.0)
    assert worst <= 1.0, what


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("requests,beams,best,vocab", [
    (1, 1, 1, 1), (1, 1, 1, 7), (1, 4, 4, 3), (3, 2, 5, 2), (1, 4, 8, 1000), (5, 3, 3, 513), (2, 8, 16, 4097), (1, 64, 64, 777),
    (7, 5, 10, 2047), (2, 1, 64, 100), (1, 2, 64, 50001), (33, 8, 8, 1111), (1, 16, 32, 200000), (600, 2, 2, 300)])
def test_select_matches_the_definition(requests, beams, best, vocab, dtype):
    x, scores = make(requests * 7 + vocab, requests, beams, vocab, dtype)
    got = run(x, scores, beams, best)
    compare(got, x, scores, beams, best, what=f"{requests}x{beams}->{best} of {vocab} {dtype}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 3), (5, 7), (8, 2)])
def test_rows_at_any_address(pad, offset, dtype):
    for vocab in (9, 1003):
        x, scores = make(pad * 10 + offset, 3, 4, vocab, dtype, pad=pad, offset=offset)
        compare(run(x, scores, 4, 6), x, scores, 4, 6, what=f"pad {pad} offset {offset}")


@pytest.mark.parametrize("requests,beams,best,vocab", [(4, 4, 4, 500), (3, 8, 16, 3001), (2, 3, 9, 4), (20, 6, 12, 901)])
def test_ended_and_dead_beams_and_weights(requests, beams, best, vocab):
    x, scores = make(vocab, requests, beams, vocab, F32)
    rng = np.random.default_rng(vocab)
    rows = requests * beams
    ended = (rng.random(rows) < 0.3).astype(np.int64)
    scores[rng.random(rows) < 0.25] = -np.inf
    ended[:beams] = 1                                   # a request that is over
    scores[beams:2 * beams] = -np.inf                   # one without beams
    scores[2 * rows // requests - 1] = np.nan
    weights = rng.random(rows).astype(np.float32) + 0.1
    weights[rng.random(rows) < 0.1] = 0.0
    weights[-1] = np.nan
    x[ended.nonzero()[0].tolist()] = math.nan                    # what is not read
    for kw in (dict(ended=ended, end_token=vocab - 1), dict(ended=ended, end_token=0, weights=weights), dict(weights=weights), dict(end_token=2)):
        y = torch.nan_to_num(x, nan=0.5) if "ended" not in kw else x
        compare(run(y, scores, beams, best, **kw), y, scores, beams, best, what=str(sorted(kw)), **kw)


def test_first_step_has_one_beam_a_request():
    x, scores = make(5, 6, 4, 2000)
    scores[:] = -np.inf
    scores[::4] = 0.0
    got = run(x, scores, 4, 4)
    compare(got, x, scores, 4, 4)
    assert (got["parents"] == np.repeat(np.arange(6) * 4, 4)).all()


@pytest.mark.parametrize("value", [0.0, -1e9, torch.finfo(BF).min, torch.finfo(BF).max, 3.0])
@pytest.mark.parametrize("best", [1, 8, 64])
def test_equal_logits_go_to_the_lowest_token_and_row(value, best):
    x, scores = make(1, 2, 8, 5003)
    x.fill_(value)
    scores[:] = -1.5
    got = run(x, scores, 8, best)
    # rows whose sums and scores are equal: the first row's tokens in order
    assert got["tokens"].tolist() == list(range(best)) * 2
    assert got["parents"].tolist() == [0] * best + [8] * best


def test_masked_vocabularies():
    """-inf and the type's lowest value at most places; fewer than `best` candidates; equal values across lists."""
    for dtype in (BF, F32):
        for low in (-math.inf, torch.finfo(dtype).min):
            x, scores = make(11, 4, 3, 9000, dtype)
            keep = torch.zeros(12, 9000, dtype=torch.bool, device="cuda")
            rng = np.random.default_rng(3)
            for r in range(12):
                keep[r, rng.choice(9000, size=r, replace=False).tolist()] = True
            x.masked_fill_(~keep, low)
            x[7, 5] = x[7, 8999] = x[7, 4000] = 1.25
            compare(run(x, scores, 3, 12), x, scores, 3, 12, what=f"masked by {low}")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_with_nan_or_infinity_give_no_candidates(bad):
    for dtype in (BF, F32):
        x, scores = make(17, 3, 4, 6000, dtype)
        for row, at in ((1, 0), (2, 5999), (6, 3001), (8, 1), (9, 2), (10, 3), (11, 4)):
            x[row, at] = bad
        got = run(x, scores, 4, 5)
        compare(got, x, scores, 4, 5, what=f"{bad}")
        assert not set(got["parents"].tolist()) & {1, 2, 6, 8, 9, 10, 11} and (got["parents"][10:] == -1).all()


def test_negative_zero_equals_zero():
    x, scores = make(2, 1, 1, 700, F32)
    x.fill_(-5.0)
    x[0, 300], x[0, 500], x[0, 600] = -0.0, 0.0, -0.0
    got = run(x, scores, 1, 3)
    assert got["tokens"].tolist() == [300, 500, 600]


@pytest.mark.parametrize("vocab", [4096, 128000])
def test_the_best_tokens_side_by_side(vocab):
    """Rows whose largest logits fill one lane's loads, in rising order: the longest lists."""
    for dtype in (BF, F32):
        x, scores = make(23, 2, 2, vocab, dtype, sigma=0.1)
        x[:, 100:700] += torch.arange(600, device="cuda").to(dtype) / 16
        compare(run(x, scores, 2, 64), x, scores, 2, 64)
        rising = (torch.arange(vocab, device="cuda") / 64.0).to(dtype)
        x.copy_(rising.expand(4, vocab))
        compare(run(x, scores, 2, 64), x, scores, 2, 64)


def test_the_result_is_the_same_on_every_call_and_stream():
    x, scores = make(31, 16, 8, 20000)
    obj = rx.Beams(0, 16, 8, 20000, 8)
    first = run(x, scores, 8, 8, obj=obj)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, None):
        again = run(x, scores, 8, 8, obj=obj, stream=stream)
        for k in first:
            assert (again[k] == first[k]).all()


def test_in_place_and_fewer_requests_than_the_object_holds():
    x, scores = make(37, 5, 4, 3000)
    ended = np.array([0, 1] * 10)
    want = run(x, scores, 4, 4, ended=ended, end_token=7)
    obj = rx.Beams(0, 9, 4, 3000)
    sc, en, par, tok = floats(scores), ints(ended), ints([0] * 20), ints([0] * 20)
    rx.beam_select(obj, x, sc, par, tok, sc, ended=en, end_token=7, ended_out=en)
    for k, v in (("parents", par), ("tokens", tok), ("scores", sc), ("ended", en)):
        assert (v.cpu().numpy() == want[k]).all(), k


def test_a_captured_selection_replays():
    x, scores = make(41, 3, 4, 8000)
    obj = rx.Beams(0, 3, 4, 8000)
    sc, out = floats(scores), Out(12)

    def call():
        rx.beam_select(obj, x, sc, out["parents"], out["tokens"], out["scores"], ended_out=out["ended"])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(4):
        y, new = make(50 + k, 3, 4, 8000)
        x.copy_(y)
        sc.copy_(floats(new))
        g.replay()
        torch.cuda.synchronize()
        compare({k: out[k].cpu().numpy() for k in out.v}, x, new, 4, 4, what="replayed")


def test_timing_names_the_launch():
    x, scores = make(1, 1, 2, 100)
    rx.lora_timing_enable(True)
    run(x, scores, 2, 2)
    report = rx.lora_timing_report()
    rx.lora_timing_enable(False)
    assert report["beam_select"][1] == 1
