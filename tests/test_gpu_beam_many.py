"""Beam selection on the GPU where a request has many candidate lists: many beams and candidates, long vocabularies."""
import numpy as np
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
from test_gpu_beam_select import BF, F32, compare, floats, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("requests,beams,best,vocab", [
    (1, 64, 64, 20000), (1, 64, 17, 60001), (1, 33, 64, 30011), (2, 40, 64, 16384), (1, 1, 64, 1000003), (1, 3, 50, 400000), (1, 16, 33, 65536),
    (5, 64, 64, 4100), (1, 64, 1, 200001)])
def test_many_lists_match_the_definition(requests, beams, best, vocab, dtype):
    x, scores = make(vocab + beams, requests, beams, vocab, dtype)
    compare(run(x, scores, beams, best), x, scores, beams, best, what=f"{requests}x{beams}->{best} of {vocab} {dtype}")


@pytest.mark.parametrize("beams,best,vocab", [(64, 64, 20000), (2, 64, 300000)])
def test_equal_logits_go_to_the_lowest_row_and_token(beams, best, vocab):
    x, _ = make(1, 1, beams, vocab, F32)
    x.zero_()
    got = run(x, np.full(beams, -1.0, dtype=np.float32), beams, best)
    assert (got["parents"] == 0).all() and (got["tokens"] == np.arange(best)).all()


@pytest.mark.parametrize("beams,best,vocab", [(64, 64, 20000), (48, 40, 30000)])
def test_one_row_has_all_of_the_best(beams, best, vocab):
    """Many lists whose best are all below one row's, and rows whose lists hold nothing."""
    x, scores = make(2, 1, beams, vocab, BF, sigma=1.0)
    scores[:] = -1000.0
    scores[beams // 2] = 0.0
    got = run(x, scores, beams, best)
    compare(got, x, scores, beams, best, what="one row")
    assert (got["parents"] == beams // 2).all()
    scores[: beams // 2] = -np.inf
    x[beams // 2, best - 3:] = -float("inf")               # fewer candidates there than places
    compare(run(x, scores, beams, best), x, scores, beams, best, what="one row and others")


@pytest.mark.parametrize("best", [5, 64])
def test_ended_and_dead_beams_and_weights(best):
    beams, vocab = 64, 20011
    x, scores = make(3, 2, beams, vocab, F32)
    rng = np.random.default_rng(best)
    rows = 2 * beams
    ended = (rng.random(rows) < 0.4).astype(np.int64)
    scores[rng.random(rows) < 0.25] = -np.inf
    weights = rng.random(rows).astype(np.float32) + 0.1
    weights[rng.random(rows) < 0.1] = 0.0
    for kw in (dict(ended=ended, end_token=vocab - 1), dict(ended=ended, end_token=0, weights=weights), dict(weights=weights)):
        compare(run(x, scores, beams, best, **kw), x, scores, beams, best, what=str(sorted(kw)), **kw)
    ended[:] = 1                                           # nothing is read any more
    compare(run(x, scores, beams, best, ended=ended, end_token=3), x, scores, beams, best, ended=ended, end_token=3, what="all ended")


def test_rising_and_falling_vocabularies():
    """The best tokens all at one end, in one or a few of the lists."""
    vocab = 500000
    up = torch.arange(vocab, device="cuda", dtype=F32) / 1000
    for x in (up, up.flip(0), (up - 250).abs(), -(up - 250).abs()):
        x = x.view(1, vocab).contiguous()
        compare(run(x, np.zeros(1, dtype=np.float32), 1, 64), x, np.zeros(1, dtype=np.float32), 1, 64, what="a slope")


def test_the_longest_vocabulary():
    vocab = rx.LORA_MAX_VOCAB
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((1, vocab), generator=g, device="cuda")
    got = run(x, np.zeros(1, dtype=np.float32), 1, 64)
    top = torch.topk(x[0], 64)
    assert (x[0][torch.from_numpy(got["tokens"]).long().cuda()] == top.values).all() and (got["parents"] == 0).all()
    want = top.values.double() - torch.logsumexp(x[0].double(), 0)
    assert (torch.from_numpy(got["scores"]).cuda().double() - want).abs().max() <= 2.0 ** -18 + 2.0 ** -24 * float(want.abs().max())


def test_an_object_for_few_lists_and_many():
    obj = rx.Beams(0, 3, 64, 20000, 64)
    for requests in (1, 3, 1, 2):
        x, scores = make(requests, requests, 64, 20000, BF)
        compare(run(x, scores, 64, 64, obj=obj), x, scores, 64, 64, what=f"{requests} requests")
    assert floats([1.0]).is_cuda
