"""Plain definitions of the paged-cache operators in 64 bits, on the CPU (test infrastructure
only; shares no code with the GPU path).  Written from the contract in include/raxlora.h:
loops over requests, tokens and heads."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["page_plan", "frequencies", "rotate", "attend", "e4m3_round"]


def page_plan(past, new, table, max_pages, ring, cursor, page, num_tokens):
    """(outputs, table, ring, cursor) of one step; inputs are not changed."""
    past, new = [int(x) for x in past], [int(x) for x in new]
    table, ring = np.array(table, dtype=np.int64), np.array(ring, dtype=np.int64)
    N = len(ring)
    head, free = int(cursor[0]) % N, min(max(int(cursor[1]), 0), N)
    ok = lambda p: 0 <= p < N  # noqa: E731
    lens, starts, pos, slots = [], [0], [], []
    asked = taken = refused = invalid = 0
    back = []
    old = table.copy()
    for r, (p, n) in enumerate(zip(past, new)):
        if p < 0 or n < -1:
            invalid += 1
            lens.append(0)
            starts.append(starts[-1])
            continue
        m = max(n, 0)
        starts.append(starts[-1] + m)
        pos += range(p, p + m)
        if p + m > max_pages * page:
            invalid += 1
            lens.append(0)
            slots += [-1] * m
            continue
        have = -(-p // page)
        if n < 0:
            back += [int(x) for x in old[r, :have]]
            lens.append(0)
            continue
        need = -(-(p + m) // page) - have
        asked += need
        if need and asked > free:
            refused += 1
            lens.append(0)
            slots += [-1] * m
            continue
        for e in range(need):
            x = int(ring[(head + taken + e) % N])
            invalid += not ok(x)
            table[r, have + e] = x if ok(x) else -1
        taken += need
        lens.append(p + m)
        for q in range(p, p + m):
            x = int(table[r, q // page])
            invalid += q // page < have and not ok(x)
            slots.append(x * page + q % page if ok(x) else -1)
    kept = back[:N - free]
    invalid += len(back) - len(kept)
    for e, x in enumerate(kept):
        invalid += not ok(x)
        ring[(head + free + e) % N] = x if ok(x) else -1
    total = starts[-1]
    invalid += max(0, total - num_tokens)
    for t in range(num_tokens, total):          # dropped tokens are only counted once
        r = next(i for i in range(len(past)) if starts[i] <= t < starts[i + 1])
        q = past[r] + t - starts[r]
        if lens[r] and q // page < -(-past[r] // page) and not ok(int(table[r, q // page])):
            invalid -= 1
    pad = max(0, num_tokens - total)
    left = free - taken + len(kept)
    return ({"seq_lens": lens, "query_start": [min(s, num_tokens) for s in starts],
             "positions": (pos + [0] * pad)[:num_tokens], "slots": (slots + [-1] * pad)[:num_tokens],
             "meta": [total, taken, len(kept), refused, invalid, left, 0, 0]},
            table, ring, [(head + taken) % N, left])


def frequencies(rot, base, scaling="plain", factor=1.0, original=0.0, low=0.0, high=0.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "wavelength":
            wavelength = 2 * math.pi / f
            if wavelength >= original / low:
                f = f / factor
            elif wavelength > original / high:
                w = (original / wavelength - low) / (high - low)
                f = (1 - w) * f / factor + w * f
        elif scaling == "dim":
            pair = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            lo, hi = min(lo, rot - 1), max(hi, 0)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return out


def rotate(x, positions, freqs, interleaved, amplitude=1.0):
    """x [T, heads, D] float64 with its first 2 len(freqs) values turned; also the size |a| +
    |b| of each turned pair times the amplitude (the bound on rounding), same shape."""
    x = np.asarray(x, dtype=np.float64)
    y, size = x.copy(), np.abs(x)
    half = len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = np.asarray(positions, dtype=np.float64) * f
        c, s = (amplitude * np.cos(ang))[:, None], (amplitude * np.sin(ang))[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def attend(q, keys, vals, table, lens, starts, page, scale, window=0):
    """q [T, H, D]; keys, vals [pages, page, KV, D] float64 -> (out, lse, bound): bound [T, H,
    D] holds sum_j p_j |v_j| and smax [T, H] the largest sum_d |q_d k_jd| scale among the keys seen."""
    T, H, D = q.shape
    N, KV = keys.shape[0], keys.shape[2]
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mass, smax = np.zeros((T, H, D)), np.zeros((T, H))
    for r in range(len(lens)):
        a, b = int(starts[r]), int(starts[r + 1])
        for t in range(a, b):
            pos = int(lens[r]) - (b - a) + (t - a)
            js = [j for j in range(max(0, pos - window + 1) if window else 0, pos + 1)
                  if 0 <= table[r][j // page] < N]
            if not js:
                continue
            pg, off = np.array([table[r][j // page] for j in js]), np.array(js) % page
            K, V = keys[pg, off], vals[pg, off]
            for h in range(H):
                k = K[:, h // (H // KV)]
                v = V[:, h // (H // KV)]
                s = k @ q[t, h] * scale
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                out[t, h] = p @ v
                lse[t, h] = m + math.log(e.sum())
                mass[t, h] = p @ np.abs(v)
                smax[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * abs(scale)
    return out, lse, mass, smax


def e4m3_round(x):
    """float64 -> the nearest e4m3 value (ties to even), clamped to [-448, 448]."""
    x = np.clip(np.asarray(x, dtype=np.float64), -448.0, 448.0)
    mag = np.abs(x)
    e = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
    step = np.exp2(np.maximum(e, -6) - 3)
    return np.where(mag > 0, np.round(x / step) * step, x)
