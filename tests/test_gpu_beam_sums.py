"""Beam selection on the GPU: log sums where every wave adds many tiles of a row."""
import math

import numpy as np
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
from lora_cases import record_error
from test_gpu_beam_select import BF, F32, HALF_STEP, LOG_SUM, floats, ints

pytestmark = pytest.mark.gpu


def check(logits, lse, best_logit, what):
    """One beam a request: scores near 0, so that their own rounding does not hide the log sums'."""
    rows, vocab = logits.shape
    obj = rx.Beams(0, rows, 1, vocab)
    scores = np.array([a - b for a, b in zip(lse, best_logit)], dtype=np.float32)
    par, tok, out = ints([-7] * rows), ints([-7] * rows), floats([7.0] * rows)
    rx.beam_select(obj, logits, floats(scores), par, tok, out)
    torch.cuda.synchronize()
    want = scores.astype(np.float64) + (np.array(best_logit) - np.array(lse))
    err = np.abs(out.cpu().numpy().astype(np.float64) - want) / (LOG_SUM + HALF_STEP * np.abs(want))
    record_error(f"log sums {what}: against their bound", "rel", float(err.max()), 1.0)
    assert (par.cpu().numpy() == np.arange(rows)).all()
    assert err.max() <= 1.0, (what, int(err.argmax()), float(err.max()))
    return tok.cpu().numpy()


@pytest.mark.parametrize("dtype,rows,vocab", [(F32, 768, 1 << 20), (BF, 768, 1 << 20), (F32, 64, 1 << 23)])
def test_equal_terms_after_a_larger_one(dtype, rows, vocab):
    """Each row's first 16384 tokens, the first tile of every wave and some more, lie above the rest, which are all equal: the
    additions of the rest all round in one direction, in every lane."""
    x = torch.zeros(rows, vocab, dtype=dtype, device="cuda")
    first, lse, top = 16384, [], []
    for r in range(rows):
        d = float(torch.tensor(0.05 + 2.9 * r / rows).to(dtype))
        x[r, :first] = d
        lse.append(math.log(first * math.exp(d) + (vocab - first)))
        top.append(d)
    assert (check(x, lse, top, f"{rows}x{vocab} {dtype}") == 0).all()


@pytest.mark.parametrize("step", [0.0, 2.0 ** -12, 2.0 ** -3])
def test_rising_rows_and_masses_far_below_the_maximum(step):
    """The maximum moves in every run or in none; most of the sum in few terms or in many small ones."""
    rows, vocab = 96, 1 << 20
    at = torch.arange(vocab, device="cuda", dtype=F32)
    x = (at // 4096 * step).expand(rows, vocab).contiguous()
    for r in range(rows):
        x[r, 777 * r + 5] += r / 6.0                       # up to 16 above its neighbours
    wide = [x[r].double() for r in range(rows)]
    lse = [float(torch.logsumexp(w, 0)) for w in wide]
    check(x, lse, [float(w.max()) for w in wide], f"step {step}")
