"""Rotary append at far positions and fast frequencies, against angles reduced in 90 decimal digits."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import rank_adapter_gemm_build_amd as rx
from test_gpu_kv import DT, E4M3, F32, HALF_STEP, act_of, f64, ints

TWO_PI = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413596429617")

POSITIONS = [2 ** 31 - 1, 2048718216, 1999999999, 2 ** 30 + 1, -(2 ** 31), -1234567891, 16777217, 1]
FREQS = [1.0, 0.7310585786300049, 1e-4, 37.25, 1.0 / 3.0, 1e5 + 1.0 / 3.0, 2.0 ** 19 + 0.1, 6.283185307179586]


def fraction(position, freq):
    """position * freq in turns, without its whole turns, exact to 2^-53 of a turn."""
    with localcontext() as c:
        c.prec = 90
        x = Decimal(position) * Decimal(freq) / TWO_PI
        return float(x - x.to_integral_value())


def test_fraction_by_hand():
    assert fraction(0, 5.0) == 0.0 and abs(fraction(1, 1.0) - 0.15915494309189535) < 2.0 ** -54
    # 355 / 113 is nearly pi: 710 radians are 113 turns and 6.03e-5 of a radian, whose sine the C library has
    assert abs(math.sin(fraction(710, 1.0) * 2 * math.pi) / math.sin(710.0) - 1) < 1e-11


@pytest.mark.gpu
@pytest.mark.parametrize("amplitude", [1.0, 1.25])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("rot", [16, 10])          # 10: a half that is no multiple of a chunk
def test_far_positions(rot, cache, inter, amplitude):
    hq, kv, dim, page, T = 4, 2, 32, 16, len(POSITIONS)
    freqs, act = FREQS[-rot // 2:], act_of(cache)
    g = torch.Generator(device="cuda")
    g.manual_seed(rot)
    qkv = torch.randn(T, (hq + 2 * kv) * dim, generator=g, device="cuda").to(act)
    k, v = (torch.zeros(1, page, kv, dim, dtype=DT[cache], device="cuda") for _ in "kv")
    q = torch.zeros(T, hq * dim, dtype=act, device="cuda")
    rx.rotary_append(rx.Rotary(0, rot, freqs, interleaved=inter, amplitude=amplitude), qkv, hq, ints(POSITIONS), ints(range(T)), q,
                     rx.KVCache(k, v))
    x = f64(qkv).reshape(T, hq + 2 * kv, dim)[:, :hq + kv]
    y, size = x.copy(), np.zeros_like(x)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        ang = [2 * math.pi * fraction(p, f) for p in POSITIONS]
        c, s = (amplitude * np.array([fn(t) for t in ang])[:, None] for fn in (math.cos, math.sin))
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = amplitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    # fp32 activations: cosine and sine rounded once, the amplitude's product, the pair's product: 2^-24 of the pair
    # each, the sum 2^-24 of the result.  16-bit ones: the fraction of a turn in fp32 (2^-26 of a turn, 2 pi 2^-26 of the
    # pair), its cosine and sine (2^-22), then the same and one rounding
    slack, half = (3.1 * 2.0 ** -24, 2.0 ** -24) if act == F32 else (2.0 ** -20, HALF_STEP[act])
    got = f64(q).reshape(T, hq, dim)
    assert (np.abs(got - y[:, :hq]) <= half * np.abs(y[:, :hq]) + slack * size[:, :hq]).all()
    got_k = f64(k)[0, :T]
    if k.dtype == E4M3:
        assert (np.abs(got_k - y[:, hq:]) <= np.maximum(2.0 ** -4 * np.abs(y[:, hq:]), 2.0 ** -10) + slack * size[:, hq:]).all()
    else:
        assert (np.abs(got_k - y[:, hq:]) <= half * np.abs(y[:, hq:]) + slack * size[:, hq:]).all()
