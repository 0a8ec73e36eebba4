"""Beam selection on the GPU with weights of infinity, which make ranks infinite, and times a score of 0 are taken as 0."""
import numpy as np
import pytest

import oracle.beam_oracle as BO
from test_gpu_beam_select import BF, F32, compare, make, run


@pytest.mark.gpu
@pytest.mark.parametrize("requests,beams,best,vocab", [(1, 2, 2, 40), (3, 8, 8, 1000), (2, 5, 12, 3), (2, 64, 64, 4100)])
def test_ended_beams_of_score_0(requests, beams, best, vocab):
    x, scores = make(vocab, requests, beams, vocab, F32)
    rows = requests * beams
    rng = np.random.default_rng(rows)
    ended = (rng.random(rows) < 0.5).astype(np.int64)
    weights = rng.random(rows).astype(np.float32) + 0.1
    weights[::beams], scores[::beams], ended[::beams] = np.inf, 0.0, 1       # rank 0, above all that are negative
    ended[1::beams] = 0
    if beams > 3:
        weights[3::beams], scores[3::beams], ended[3::beams] = np.inf, -0.0, 1
        weights[4::beams], scores[4::beams], ended[4::beams] = np.inf, 2.0, 1   # rank +inf: the first of all
    got = run(x, scores, beams, best, ended=ended, end_token=0, weights=weights)
    compare(got, x, scores, beams, best, ended=ended, end_token=0, weights=weights, what="infinite weights")
    first = np.arange(requests) * beams
    want = [[f] for f in first] if beams <= 3 else [[f + 4, f, f + 3] for f in first]
    for r, w in enumerate(want):
        assert got["parents"][r * best:r * best + len(w)].tolist() == w


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("requests,beams,best,vocab", [(1, 1, 4, 100), (2, 4, 4, 3000), (1, 64, 64, 20000)])
def test_rows_with_weights_of_infinity(requests, beams, best, vocab, dtype):
    """Where no beam has ended: ranks of minus infinity, in order of rows and logits, and one of 0 where a token has all the mass."""
    x, scores = make(vocab, requests, beams, vocab, dtype)
    rows = requests * beams
    weights = np.full(rows, np.inf, dtype=np.float32)
    compare(run(x, scores, beams, best, weights=weights), x, scores, beams, best, weights=weights, what="all infinite")
    scores[-1] = 0.0
    x[-1, 7] = 2000.0                                                        # s = 0 there, and the others -2000 or so
    got = run(x, scores, beams, best, weights=weights)
    compare(got, x, scores, beams, best, weights=weights, what="one has all the mass")
    assert got["parents"][-best] == rows - 1 and got["tokens"][-best] == 7


def test_the_definition():
    got = BO.select([[0.0, 1.0], [0.0, 1.0]], [0.0, -1.0], 2, 4, ended=[1, 1], end_token=1, weights=[np.inf, 1.0])
    assert [(r, t) for _, r, t, _, _ in got[0]] == [(0, 1), (1, 1)]
