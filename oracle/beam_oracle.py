"""Plain definitions of the operators of beam search over the paged cache in 64 bits, on the CPU (test infrastructure
only; shares no code with the GPU path).  Written from the contract in include/raxlora.h: loops over rows,
candidates and pages."""
from __future__ import annotations

import math

import numpy as np

__all__ = ["log_sums", "select", "page_fork", "page_copy"]


def log_sums(logits):
    """ln sum exp of each row; NaN where a row holds NaN or +inf, -inf where it has no finite value."""
    out = []
    for x in np.asarray(logits, dtype=np.float64):
        if np.isnan(x).any() or (x == np.inf).any():
            out.append(math.nan)
            continue
        top = x.max()
        out.append(top + math.log(np.exp(x - top).sum()) if top > -np.inf else -math.inf)
    return out


def select(logits, scores, beams, best, ended=None, end_token=-1, weights=None):
    """Per request the ranked candidates [(rank, row, token, score, ended)], at most `best` of them."""
    x = np.asarray(logits, dtype=np.float64)
    lse = log_sums(x)
    rank = lambda s, w: s * w if s else 0.0  # noqa: E731  (infinity times 0 is taken as 0)
    out = []
    for r in range(x.shape[0] // beams):
        found = []
        for row in range(r * beams, (r + 1) * beams):
            c, w = float(scores[row]), 1.0 if weights is None else float(weights[row])
            if not c > -math.inf or not w > 0:
                continue
            if ended is not None and ended[row]:
                found.append((rank(c, w), row, 0, int(end_token), c, 1))
                continue
            if not math.isfinite(lse[row]):
                continue
            order = np.lexsort((np.arange(x.shape[1]), -x[row]))[:best]        # larger logit, then lower token
            for place, t in enumerate(order):
                if x[row, t] > -math.inf:
                    s = c + (x[row, t] - lse[row])
                    found.append((rank(s, w), row, place, int(t), s, int(t == end_token)))
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        out.append([(f[0], f[1], f[3], f[4], f[5]) for f in found[:best]])
    return out


def page_fork(parents, lens, table, max_pages, ring, cursor, shares, page):
    """(outputs, lens, table, ring, cursor, shares) after the call; inputs are not changed."""
    R, N = len(parents), len(ring)
    ok = lambda p: 0 <= p < N  # noqa: E731
    old = np.array(table, dtype=np.int64)
    table, ring, shares = old.copy(), [int(x) for x in ring], [int(x) for x in shares]
    head, free = int(cursor[0]) % N, min(max(int(cursor[1]), 0), N)
    invalid, size = 0, []
    for n in lens:
        good = 0 <= n <= max_pages * page
        invalid += not good
        size.append(int(n) if good else 0)
    par = []
    for p in parents:
        invalid += not -1 <= p < R
        par.append(int(p) if 0 <= p < R else -1)
    src, dst, tokens = [-1] * R, [-1] * R, [0] * R
    kids, new, seen = [0] * R, [0] * R, set()
    asked = taken = 0
    drawn = []
    for i, p in enumerate(par):
        if p < 0:
            continue
        part = size[p] % page
        if part and p in seen:
            asked += 1
            if asked > free:
                continue
            drawn.append((i, p, taken))
            taken += 1
        seen.add(p)
        kids[p] += 1
        new[i] = size[p]
        for c in range(-(-size[p] // page)):
            table[i, c] = old[p, c] if ok(old[p, c]) else -1
    for i, p, n in drawn:
        at = size[p] // page
        fresh = ring[(head + n) % N]
        invalid += not ok(fresh)
        table[i, at] = fresh if ok(fresh) else -1
        if ok(fresh) and ok(old[p, at]):
            src[i], dst[i], tokens[i] = int(old[p, at]), fresh, size[p] % page
    freed = set()
    for r in range(R):
        for c in range(-(-size[r] // page)):
            p = int(old[r, c])
            if not ok(p):
                invalid += 1
                continue
            shares[p] += kids[r] - 1 if c < size[r] // page else -(kids[r] == 0)
    for p in range(N):
        if shares[p] < 0:
            freed.add(p)
            shares[p] = 0
    back = sorted(freed)
    kept = back[:N - free]
    invalid += len(back) - len(kept)
    for e, p in enumerate(kept):
        ring[(head + free + e) % N] = p
    left = free - taken + len(kept)
    return ({"copy_src": src, "copy_dst": dst, "copy_tokens": tokens, "meta": [taken, len(kept), asked - taken, invalid, left, 0, 0, 0]},
            new, table, ring, [(head + taken) % N, left], shares)


def page_copy(cells, src, dst, tokens, page):
    """cells [pages, page, ...] after the copies."""
    out = np.array(cells)
    N = out.shape[0]
    for i, (a, b) in enumerate(zip(src, dst)):
        if 0 <= a < N and 0 <= b < N and a != b:
            n = page if tokens is None else min(max(int(tokens[i]), 0), page)
            out[b, :n] = cells[a, :n]
    return out

