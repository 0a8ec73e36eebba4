"""The operators of beam search and of batches with a common prefix over a paged cache, as measured cases.

Four operators, in the order a step uses them:

  select  the best continuations of every request over its beams and the vocabulary, from the logits
  fork    block table rows that follow their beams: pages shared, partly filled ones drawn anew, unused ones given back
  copy    the cells of the pages that a fork has to copy, in all layers of the cache
  shared  attention of sequences that have their first tokens in common pages, which are read once for all of them

With ``own`` false, ``run`` computes the plain form in elementary torch operations; with ``own``
true it makes the calls of rank_adapter_gemm_build_amd.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": E4M3}
SIZES = {"bf16": 2, "f32": 4, "fp8": 1}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request with four beams: the smallest step, bound by latency
        {"name": "select-1x4", "op": "select", "requests": 1, "beams": 4, "best": 4, "vocab": 32000, "type": "bf16",
         "ended": 0, "dead": 0, "weights": False, "pad": 0},
        # 24 requests with six beams and a spare candidate for each, some beams over, ranked by length; rows at odd addresses
        {"name": "select-24x6-f32", "op": "select", "requests": 24, "beams": 6, "best": 12, "vocab": 50001, "type": "f32",
         "ended": 20, "dead": 7, "weights": True, "pad": 0},
        # a full step: 64 requests with eight beams over a large vocabulary
        {"name": "select-64x8", "op": "select", "requests": 64, "beams": 8, "best": 8, "vocab": 128000, "type": "bf16",
         "ended": 0, "dead": 0, "weights": False, "pad": 0},
        # four beams of one request
        {"name": "fork-1x4", "op": "fork", "requests": 1, "beams": 4, "len_lo": 777, "len_hi": 777, "grown": 60, "ended": 0,
         "page": 16, "short": 0},
        # 128 requests with eight beams, eleven of which have just ended and give their pages back
        {"name": "fork-128x8", "op": "fork", "requests": 128, "beams": 8, "len_lo": 100, "len_hi": 8191, "grown": 500,
         "ended": 11, "page": 16, "short": 0},
        # the pages that four beams copy in a step, in 32 layers
        {"name": "copy-3x32", "op": "copy", "pairs": 3, "layers": 32, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16,
         "order": "token", "whole": False},
        # whole pages of an 8-bit cache whose heads lie apart
        {"name": "copy-200x8-fp8", "op": "copy", "pairs": 200, "layers": 8, "kv_heads": 8, "dim": 128, "cache": "fp8",
         "page": 64, "order": "head", "whole": True},
        # the pages that 64 requests with eight beams copy in a step, in 32 layers
        {"name": "copy-448x32", "op": "copy", "pairs": 448, "layers": 32, "kv_heads": 8, "dim": 128, "cache": "bf16",
         "page": 16, "order": "token", "whole": False},
        # four beams over one prompt: latency
        {"name": "shared-1x4", "op": "shared", "groups": 1, "members": 4, "common_lo": 704, "common_hi": 704, "own_lo": 20,
         "own_hi": 70, "new": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16, "order": "token",
         "idle": 0, "ragged": False},
        # 24 requests with eight beams over an 8-bit cache; two beams are over
        {"name": "shared-24x8-fp8", "op": "shared", "groups": 24, "members": 8, "common_lo": 1000, "common_hi": 6000,
         "own_lo": 1, "own_hi": 300, "new": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "cache": "fp8", "page": 64,
         "order": "token", "idle": 2, "ragged": False},
        # 64 chats that begin with the same instructions
        {"name": "shared-64-8000", "op": "shared", "groups": 1, "members": 64, "common_lo": 8000, "common_hi": 8000,
         "own_lo": 10, "own_hi": 900, "new": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16,
         "order": "token", "idle": 0, "ragged": False},
        # a full server: 256 chats about one long document
        {"name": "shared-256-32000", "op": "shared", "groups": 1, "members": 256, "common_lo": 32000, "common_hi": 32000,
         "own_lo": 100, "own_hi": 2000, "new": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16,
         "order": "token", "idle": 0, "ragged": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "copy", "shared", "shared", "shared"])
    if op == "select":
        kind = rng.choice(["bf16", "bf16", "f32"])
        beams = rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 16])
        vocab = rng.choice([_log_int(rng, 300, 200000), 8 * _log_int(rng, 1000, 20000)])
        requests = _log_int(rng, 1, max(1, min(256, 130_000_000 // (beams * vocab * SIZES[kind]))))
        rows = requests * beams
        return {"op": op, "requests": requests, "beams": beams, "best": rng.choice([beams, beams, 2 * beams]), "vocab": vocab,
                "type": kind, "ended": rng.randint(0, rows // 3), "dead": rng.randint(0, rows // 4),
                "weights": rng.random() < 0.5, "pad": rng.choice([0, 0, rng.randint(1, 64)])}
    if op == "fork":
        beams = rng.choice([1, 2, 3, 4, 8, 8, 16])
        requests = _log_int(rng, 1, 1024 // beams)
        len_hi = _log_int(rng, 4, 8192)
        return {"op": op, "requests": requests, "beams": beams, "len_lo": rng.randint(1, len_hi), "len_hi": len_hi,
                "grown": rng.randint(1, 600), "ended": rng.randint(0, requests // 4), "page": rng.choice([16, 32, 64, 128]),
                "short": rng.choice([0, 0, rng.randint(1, 20)])}
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    cache = rng.choice(["bf16", "bf16", "fp8", "f32"])
    page, order = rng.choice([16, 32, 64, 128]), rng.choice(["token", "head"])
    if op == "copy":
        layers = rng.randint(1, 40)
        cells = 2 * layers * page * kv_heads * dim * SIZES[cache]      # bytes of a page in all layers
        return {"op": op, "pairs": _log_int(rng, 1, max(1, min(1024, 400_000_000 // cells))), "layers": layers,
                "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page, "order": order, "whole": rng.random() < 0.3}
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 8])
    row = 2 * kv_heads * dim * SIZES[cache]                            # bytes of one token in the cache
    members = _log_int(rng, 1, 128)
    groups = _log_int(rng, 1, max(1, 128 // members))
    own_hi = _log_int(rng, 1, min(2000, max(1, 400_000_000 // (row * members * groups))))
    most = min(20000, 400_000_000 // (row * groups), 400_000_000 // (groups * members * kv_heads * group))
    common_hi = _log_int(rng, page, max(page, most))
    return {"op": op, "groups": groups, "members": members, "common_lo": rng.randint(0, common_hi), "common_hi": common_hi,
            "own_lo": rng.randint(1, own_hi), "own_hi": own_hi, "new": rng.choice([1, 1, 1, 2, 4]), "q_heads": kv_heads * group,
            "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page, "order": order,
            "idle": rng.choice([0, 1]) if members > 1 else 0, "ragged": rng.random() < 0.5}


# ------------------------------------------------------------------------------------ sizes that follow from a case
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _ceil(a, b):
    return -(-a // b)


def _act(case):
    return "f32" if case["cache"] == "f32" else "bf16"


def _fork_lens(case):
    """(cached length, tokens since the beams began) of every request."""
    lens = _spread(case["len_lo"], case["len_hi"], case["requests"])
    return lens, [min(n, max(1, case["grown"] * (i % 5 + 1) // 5)) for i, n in enumerate(lens)]


def _copy_tokens(case):
    """Tokens of each pair's page."""
    p = case["page"]
    return [p if case["whole"] else 1 + 7 * i % (p - 1) for i in range(case["pairs"])]


def _shared_sizes(case):
    """Per group its common tokens and its members' own; `ragged` groups have from one member to all."""
    n, m = case["groups"], case["members"]
    common = _spread(case["common_lo"], case["common_hi"], n)
    sizes = [1 + (i * 5 + m - 1) % m for i in range(n)] if case["ragged"] else [m] * n
    if not case["ragged"]:                                             # whole pages, as a fork leaves them
        common = [c // case["page"] * case["page"] for c in common]
    own_ = _spread(case["own_lo"], case["own_hi"], sum(sizes))
    return common, sizes, [own_[(i * 11) % len(own_)] for i in range(len(own_))]


def work(case):
    if case["op"] == "select":
        rows, v = case["requests"] * case["beams"], case["vocab"]
        read = rows - case["ended"] - case["dead"]
        return {"bytes": read * v * SIZES[case["type"]] + 12 * rows + 16 * case["requests"] * case["best"], "flops": 4 * read * v}
    if case["op"] == "fork":
        lens, _ = _fork_lens(case)
        entries = case["beams"] * sum(_ceil(n, case["page"]) for n in lens)
        rows = case["requests"] * case["beams"]
        return {"bytes": 8 * entries + 24 * rows, "flops": entries}
    d = case["kv_heads"] * case["dim"] * SIZES[case["cache"]]
    if case["op"] == "copy":
        return {"bytes": 4 * case["layers"] * sum(_copy_tokens(case)) * d + 12 * case["pairs"], "flops": 0}
    common, sizes, own_ = _shared_sizes(case)
    new, tokens = case["new"], case["new"] * len(own_)
    pairs = sum(c * s for c, s in zip(common, sizes)) * new + sum(own_) * new
    return {"bytes": 2 * (sum(common) + sum(own_)) * d + 2 * tokens * case["q_heads"] * case["dim"] * SIZES[_act(case)]
            + 4 * tokens * case["q_heads"] + 4 * _ceil(sum(common) + sum(own_), case["page"]),
            "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ------------------------------------------------------------------------------------ inputs
def _int32(values):
    return torch.from_numpy(np.asarray(values, dtype=np.int64).astype(np.int32)).cuda()


def _fill(x, gen):
    """Normal values, a part at a time."""
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return x


def _cache(case, pages, gen, layers=None):
    """Keys or values ([layers,] pages, page, heads, dim) in the order of the case."""
    kv, d, p = case["kv_heads"], case["dim"], case["page"]
    shape = (pages, p, kv, d) if case["order"] == "token" else (pages, kv, p, d)
    x = _fill(torch.empty(shape if layers is None else (layers, *shape), dtype=DTYPES[case["cache"]], device="cuda"), gen)
    return x if case["order"] == "token" else x.transpose(-3, -2)


def _select_inputs(case, rng, gen, s):
    rows, v = case["requests"] * case["beams"], case["vocab"]
    logits = torch.empty((rows, v + case["pad"]), dtype=DTYPES[case["type"]], device="cuda")
    for i in range(0, rows, 256):                                      # a language model's: wide, each row at its own level
        part = logits[i:i + 256]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * 3.0
                   + torch.randn((part.shape[0], 1), generator=gen, device="cuda"))
    logits[:, v:] = math.nan                                           # behind a row lies what is not read
    order = list(range(rows))
    rng.shuffle(order)
    ended, scores = np.zeros(rows, dtype=np.int64), np.array([-rng.uniform(0.0, 12.0) for _ in range(rows)])
    ended[order[:case["ended"]]] = 1
    scores[order[case["ended"]:case["ended"] + case["dead"]]] = -math.inf
    s.update(logits=logits[:, :v], scores=torch.from_numpy(scores.astype(np.float32)).cuda(),
             ended=_int32(ended) if case["ended"] else None, end_token=rng.randrange(v) if case["ended"] else -1,
             weights=torch.tensor([(rng.randint(5, 60)) ** -0.6 for _ in range(rows)], device="cuda") if case["weights"] else None)
    n = case["requests"] * case["best"]
    s["out"] = {"parents": _int32(np.zeros(n)), "tokens": _int32(np.zeros(n)), "scores": torch.zeros(n, device="cuda"),
                "ended": _int32(np.zeros(n))}


def _fork_inputs(case, rng, gen, s):
    p, w = case["page"], case["beams"]
    lens, grown = _fork_lens(case)
    order = list(range(case["requests"]))
    rng.shuffle(order)
    gone = set(rng.sample(order, case["ended"]))
    width = max(_ceil(n, p) for n in lens) + 2
    table = np.full((case["requests"] * w, width), -1, dtype=np.int64)
    holders, parents, at, extra = [], [], 0, 0
    for place, r in enumerate(order):
        full, begun = lens[r] // p, (lens[r] - grown[r]) // p          # full pages; those before the beams
        rows = slice(place * w, place * w + w)
        for c in range(_ceil(lens[r], p)):
            # beams that have the same history so far share a page; the partly filled last one is each beam's own
            n = 1 if c < begun else w if c >= full else min(w, 1 + (c - begun) * w // max(1, full - begun))
            table[rows, c] = at + np.arange(w) * n // w
            holders += np.bincount(np.arange(w) * n // w, minlength=n).tolist()
            at += n
        mine = [-1] * w if r in gone else [place * w + rng.randrange(w) for _ in range(w)]
        parents += mine
        extra += (w - len(set(mine))) * (lens[r] % p > 0) if r not in gone else 0
    free = max(0, extra - case["short"]) if case["short"] else extra + 5
    pages = at + len(parents) + 5                                      # those neither held here nor free are held elsewhere
    ids = np.random.default_rng(rng.randrange(1 << 30)).permutation(pages)
    ring = np.full(pages, -1, dtype=np.int64)
    head = rng.randrange(pages)
    ring[(head + np.arange(free)) % pages] = ids[at:at + free]
    shares = np.zeros(pages, dtype=np.int64)
    shares[ids[:at]] = np.array(holders) - 1
    s.update(parents=_int32(parents), lens=_int32([lens[r] for r in order for _ in range(w)]), pages=pages,
             table=_int32(np.where(table >= 0, ids[table], -1)), ring=_int32(ring), cursor=_int32([head, free, 0, 0]),
             shares=_int32(shares))
    s["out"] = {k: _int32(np.zeros(len(parents))) for k in ("copy_src", "copy_dst", "copy_tokens")}


def _copy_inputs(case, rng, gen, s):
    n, layers = case["pairs"], case["layers"]
    pages = 2 * n + 3
    ids = list(range(pages))
    rng.shuffle(ids)
    tokens = _copy_tokens(case)
    rng.shuffle(tokens)
    src = [ids[rng.randrange(n)] for _ in range(n)]                    # several copies of one page among them
    s.update(k=_cache(case, pages, gen, layers), v=_cache(case, pages, gen, layers), src=_int32(src), dst=_int32(ids[n:2 * n]),
             tokens=None if case["whole"] else _int32(tokens))


def _shared_inputs(case, rng, gen, s):
    p, new = case["page"], case["new"]
    common, sizes, own_ = _shared_sizes(case)
    n = len(own_)
    # tokens of a sequence: the common ones and its own, the new ones among them
    lens = [c + max(x, new) for c, x in zip([c for c, m in zip(common, sizes) for _ in range(m)], own_)]
    starts, group_start = [0], [0]
    for m in sizes:
        group_start.append(group_start[-1] + m)
    for _ in lens:
        starts.append(starts[-1] + new)
    pages = sum(_ceil(c, p) for c in common) + sum(_ceil(x, p) for x in lens)
    ids = np.random.default_rng(rng.randrange(1 << 30)).permutation(pages)
    table = np.full((n, max(_ceil(x, p) for x in lens) + 1), -1, dtype=np.int64)
    at = 0
    for g, (c, m) in enumerate(zip(common, sizes)):
        both = ids[at:at + _ceil(c, p)]
        at += len(both)
        for i in range(group_start[g], group_start[g] + m):
            rest = _ceil(lens[i], p) - len(both)
            table[i, :len(both) + rest] = np.concatenate([both, ids[at:at + rest]])
            at += rest
    for i in rng.sample(range(n), case["idle"]):
        lens[i] = 0
    t, act = n * new, DTYPES[_act(case)]
    width = case["q_heads"] * case["dim"]
    s.update(q=(torch.randn((t, width), generator=gen, device="cuda") * 1.5).to(act), k=_cache(case, pages, gen),
             v=_cache(case, pages, gen), scales=(0.75, 1.25) if case["cache"] == "fp8" else (1.0, 1.0), table=_int32(table),
             lens=_int32(lens), starts=_int32(starts), group_start=_int32(group_start), common=_int32(common),
             most_common=max(common), most_own=max(max(own_), new), most_members=max(sizes), scale=1.0 / math.sqrt(case["dim"]),
             out=torch.zeros((t, width), dtype=act, device="cuda"),
             lse=torch.zeros((t, case["q_heads"]), dtype=torch.float32, device="cuda"))


def _inputs(case, seed):
    rng, gen = random.Random(seed), torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    {"select": _select_inputs, "fork": _fork_inputs, "copy": _copy_inputs, "shared": _shared_inputs}[case["op"]](case, rng, gen, s)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import rank_adapter_gemm_build_amd as rx
        if case["op"] == "select":
            s["beams"] = rx.Beams(0, case["requests"], case["beams"], case["vocab"], case["best"])
        elif case["op"] == "fork":
            s["plan"] = rx.ForkPlan(0, case["requests"] * case["beams"], s["pages"])
        elif case["op"] == "copy":
            s["kv"] = rx.KVLayers([rx.KVCache(k, v) for k, v in zip(s["k"], s["v"])])
        else:
            s["kv"] = rx.KVCache(s["k"], s["v"], *s["scales"])
            s["attention"] = rx.SharedAttention(0, len(s["lens"]), s["q"].shape[0], case["q_heads"], case["kv_heads"], case["dim"])
    return s


# ------------------------------------------------------------------------------------ plain forms
def _plain_select(s):
    c, out = s["case"], s["out"]
    w, k, v = c["beams"], c["best"], c["vocab"]
    x, score = s["logits"].double(), s["scores"].double()[:, None]     # 64 bits: candidates of two beams can lie next to each other
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    cand = score + (x - lse)
    if s["ended"] is not None:
        over, same = s["ended"][:, None] != 0, torch.arange(v, device=x.device) == s["end_token"]
        cand = torch.where(over, torch.where(same, score, -math.inf), cand)
    cand = torch.where((score > -math.inf) & (cand > -math.inf), cand, -math.inf)
    rank = cand if s["weights"] is None else cand * s["weights"].double()[:, None]
    place = rank.view(-1, w * v).sort(dim=-1, descending=True, stable=True)[1][:, :k]
    best = cand.view(-1, w * v).gather(1, place)
    there = best > -math.inf
    row = torch.arange(c["requests"], device=x.device)[:, None] * w + place // v
    out["parents"].copy_(torch.where(there, row, -1).view(-1))
    out["tokens"].copy_(torch.where(there, place % v, -1).view(-1))
    out["scores"].copy_(best.view(-1))
    done = place % v == s["end_token"]
    if s["ended"] is not None:
        done = done | (s["ended"][row] != 0)
    out["ended"].copy_((there & done).view(-1))
    return out


def _plain_fork(s):
    p, pages, out = s["case"]["page"], s["pages"], s["out"]
    par, lens, table, ring, shares = s["parents"].long(), s["lens"].long(), s["table"], s["ring"], s["shares"]
    head, free = s["cursor"][0].long(), s["cursor"][1].long()
    n = par.shape[0]
    rows, col = torch.arange(n, device=par.device), torch.arange(table.shape[1], device=par.device)
    has, up = par >= 0, par.clamp(min=0)
    size = torch.where(has, lens[up], 0)
    # the first to follow a row keeps its partly filled page, the others draw one
    first = torch.full((n + 1,), n, device=par.device).scatter_reduce(0, torch.where(has, par, n), rows, "amin")
    need = has & (first[up] != rows) & (size % p > 0)
    rank = need.long().cumsum(0) - need.long()
    granted = has & (~need | (rank < free))
    draws = need & granted
    taken = draws.sum()
    kids = torch.zeros(n + 1, dtype=torch.long, device=par.device).scatter_add(0, torch.where(granted, par, n), torch.ones_like(par))[:n, None]
    # holders of the pages
    held, full = col < ((lens + p - 1) // p)[:, None], col < (lens // p)[:, None]
    change = torch.where(full, kids - 1, torch.where(kids > 0, 0, -1)).expand_as(held)
    shares.scatter_add_(0, table[held].long(), change[held].int())
    freed = shares < 0
    ring[((head + free + freed.long().cumsum(0) - 1) % pages)[freed]] = torch.arange(pages, device=par.device)[freed].int()
    shares.clamp_(min=0)
    # rows
    tail = size // p
    fresh = ring[(head + rank) % pages]
    old = table[up, tail.clamp(max=table.shape[1] - 1)]
    moved = torch.where(draws[:, None] & (col == tail[:, None]), fresh[:, None], table[up])
    table.copy_(torch.where(granted[:, None] & (col < ((size + p - 1) // p)[:, None]), moved, table))
    out["copy_src"].copy_(torch.where(draws, old, -1))
    out["copy_dst"].copy_(torch.where(draws, fresh, -1))
    out["copy_tokens"].copy_(torch.where(draws, size % p, 0))
    s["lens"].copy_(torch.where(granted, size, 0))
    s["cursor"][:2] = torch.stack([(head + taken) % pages, free - taken + freed.sum()]).int()
    return {"table": table, "lens": s["lens"], "shares": shares, "free_pages": ring, "cursor": s["cursor"], **out}


def _plain_copy(s):
    p, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    bytes_ = (lambda x: x.view(torch.uint8)) if s["case"]["cache"] == "fp8" else (lambda x: x)
    for x in (bytes_(s["k"]), bytes_(s["v"])):
        if s["tokens"] is None:
            x[:, dst] = x[:, src]
        else:
            use = (torch.arange(p, device=src.device) < s["tokens"][:, None])[None, :, :, None, None]
            x[:, dst] = torch.where(use, x[:, src], x[:, dst])
    return {"k": s["k"], "v": s["v"]}


def _plain_shared(s):
    c = s["case"]
    h, kv, d, p, new = c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["new"]
    g, n, groups = h // kv, len(s["lens"]), len(s["common"])
    lens, starts, bounds, common = s["lens"].long(), s["starts"].long(), s["group_start"].long(), s["common"].long()
    table, dev = s["table"].long(), s["lens"].device
    bytes_ = (lambda x: x.view(torch.uint8)) if c["cache"] == "fp8" else (lambda x: x)
    cells = lambda x, page, at, scale: bytes_(x)[page, at].view(x.dtype).float() * scale  # noqa: E731
    seq = torch.arange(n, device=dev)
    of = torch.searchsorted(bounds, seq, right=True) - 1                            # the group of each sequence
    count = starts[1:] - starts[:-1]
    part = (lens > 0) & (lens - count >= common[of])                                # sequences that read the common tokens
    lead = torch.full((groups,), n, device=dev).scatter_reduce(0, of, torch.where(part, seq, n), "amin").clamp(max=n - 1)
    tok = torch.arange(s["q"].shape[0], device=dev)
    tseq = torch.searchsorted(starts, tok, right=True) - 1
    q = s["q"].float().view(-1, kv, g, d)
    # common tokens: a group's rows together
    m = s["most_members"] * new
    tgroup = of[tseq]
    at = tok - starts[bounds[tgroup]]
    rows = torch.zeros((groups, m, kv, g, d), device=dev)
    rows[tgroup, at] = q
    rows = rows.permute(0, 2, 1, 3, 4).reshape(groups, kv, m * g, d)
    j = torch.arange(max(1, s["most_common"]), device=dev)
    page = table[lead][:, j // p].clamp(min=0)
    keys, vals = (cells(x, page, j % p, y).permute(0, 2, 1, 3).contiguous() for x, y in ((s["k"], s["scales"][0]), (s["v"], s["scales"][1])))
    a = torch.matmul(rows, keys.transpose(2, 3).contiguous()).view(groups, kv, m, g, -1).permute(0, 2, 1, 3, 4)[tgroup, at] * s["scale"]
    a = a.masked_fill(~(part[tseq][:, None] & (j < common[tgroup][:, None]))[:, None, None], -math.inf)
    # own tokens: a sequence's rows together
    base = torch.where(part, common[of], 0)
    i = torch.arange(max(1, s["most_own"]), device=dev)
    pos = base[:, None] + i
    page = table.gather(1, (pos // p).clamp(max=table.shape[1] - 1)).clamp(min=0)
    okeys, ovals = (cells(x, page, pos % p, y).permute(0, 2, 1, 3).contiguous() for x, y in ((s["k"], s["scales"][0]), (s["v"], s["scales"][1])))
    mine = q.view(n, new, kv, g, d).permute(0, 2, 1, 3, 4).reshape(n, kv, new * g, d)
    b = torch.matmul(mine, okeys.transpose(2, 3).contiguous()).view(n, kv, new, g, -1).permute(0, 2, 1, 3, 4).reshape(-1, kv, g, len(i)) * s["scale"]
    place = (lens - count)[tseq] + tok - starts[tseq]
    b = b.masked_fill(~((pos[tseq] <= place[:, None]) & (pos < lens[:, None])[tseq])[:, None, None], -math.inf)
    # softmax over both
    top = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    low = top.masked_fill(top == -math.inf, 0.0)
    a, b = (a - low).exp(), (b - low).exp()
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    wide = torch.zeros((groups, m, kv, g, len(j)), device=dev)
    wide[tgroup, at] = a
    o = torch.matmul(wide.permute(0, 2, 1, 3, 4).reshape(groups, kv, m * g, len(j)), vals)
    o = o.view(groups, kv, m, g, d).permute(0, 2, 1, 3, 4)[tgroup, at]
    u = torch.matmul(b.view(n, new, kv, g, -1).permute(0, 2, 1, 3, 4).reshape(n, kv, new * g, -1), ovals)
    o = o + u.view(n, kv, new, g, d).permute(0, 2, 1, 3, 4).reshape(-1, kv, g, d)
    s["out"].copy_((o / total.clamp(min=1e-38)).reshape(-1, h * d))
    s["lse"].copy_((top + total.log()).reshape(-1, h))
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"select": _plain_select, "fork": _plain_fork, "copy": _plain_copy, "shared": _plain_shared}[op](s)
    import rank_adapter_gemm_build_amd as rx
    if op == "select":
        out = s["out"]
        rx.beam_select(s["beams"], s["logits"], s["scores"], out["parents"], out["tokens"], out["scores"], ended=s["ended"],
                       end_token=s["end_token"], ended_out=out["ended"], weights=s["weights"])
        return out
    if op == "fork":
        plan = s["plan"]
        rx.page_fork(plan, s["parents"], s["lens"], s["ring"], s["cursor"], s["shares"], s["table"], s["case"]["page"])
        return {"table": s["table"], "lens": s["lens"], "shares": s["shares"], "free_pages": s["ring"], "cursor": s["cursor"],
                "copy_src": plan.copy_src, "copy_dst": plan.copy_dst, "copy_tokens": plan.copy_tokens}
    if op == "copy":
        rx.page_copy(s["kv"], s["src"], s["dst"], s["tokens"])
        return {"k": s["k"], "v": s["v"]}
    rx.shared_attention(s["attention"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], s["group_start"], s["common"], s["out"],
                        scale=s["scale"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------ the definitions, in 64 bits
def _exact_select(s):
    c = s["case"]
    w, k = c["beams"], c["best"]
    scores = s["scores"].double().tolist()
    ended = s["ended"].tolist() if s["ended"] is not None else [0] * len(scores)
    weight = s["weights"].double().tolist() if s["weights"] is not None else [1.0] * len(scores)
    parents, tokens, best, done = [], [], [], []
    for r in range(c["requests"]):
        found = []
        for row in range(r * w, r * w + w):
            if scores[row] == -math.inf:
                continue
            if ended[row]:
                found.append((-scores[row] * weight[row], row, s["end_token"], scores[row]))
                continue
            x = s["logits"][row].double()
            lse = float(torch.logsumexp(x, 0))
            # the row's k largest logits, the lower token first among equal ones
            least = x.kthvalue(max(1, x.numel() - k + 1)).values if x.numel() > k else x.min()
            near = (x >= least).nonzero()[:, 0]
            for y, t in sorted(zip((-x[near]).tolist(), near.tolist()))[:k]:
                z = scores[row] + (-y - lse)
                found.append((-z * weight[row], row, t, z))
        found = sorted(found)[:k]
        found += [(0.0, -1, -1, -math.inf)] * (k - len(found))
        parents += [f[1] for f in found]
        tokens += [f[2] for f in found]
        best += [f[3] for f in found]
        done += [int(f[1] >= 0 and (ended[f[1]] != 0 or f[2] == s["end_token"])) for f in found]
    return {"parents": _int32(parents), "tokens": _int32(tokens), "ended": _int32(done),
            "scores": torch.tensor(best, dtype=torch.float64, device="cuda")}


def _exact_fork(s):
    p, pages = s["case"]["page"], s["pages"]
    par, lens, old = s["parents"].tolist(), s["lens"].tolist(), s["table"].cpu().numpy()
    ring, shares, table = s["ring"].cpu().numpy().copy(), s["shares"].cpu().numpy().copy(), old.copy()
    head, free = s["cursor"].tolist()[:2]
    kept, kids, size, taken = set(), [0] * len(par), [0] * len(par), 0
    src, dst, tokens = ([-1] * len(par), [-1] * len(par), [0] * len(par))
    asked = 0
    for i, r in enumerate(par):
        if r < 0:
            continue
        if lens[r] % p and r in kept:
            asked += 1
            if asked > free:
                continue
            page = ring[(head + taken) % pages]
            taken += 1
            src[i], dst[i], tokens[i] = old[r, lens[r] // p], page, lens[r] % p
        kept.add(r)
        kids[r] += 1
        size[i] = lens[r]
        n = _ceil(lens[r], p)
        table[i, :n] = old[r, :n]
        if dst[i] >= 0:
            table[i, n - 1] = dst[i]
    for r, n in enumerate(lens):
        for c in range(_ceil(n, p)):
            shares[old[r, c]] += kids[r] - 1 if c < n // p else (0 if kids[r] else -1)
    back = [int(x) for x in np.flatnonzero(shares < 0)]
    for e, x in enumerate(back):
        ring[(head + free + e) % pages] = x
        shares[x] = 0
    return {"table": _int32(table), "lens": _int32(size), "shares": _int32(shares), "free_pages": _int32(ring),
            "cursor": _int32([(head + taken) % pages, free - taken + len(back), 0, 0]), "copy_src": _int32(src),
            "copy_dst": _int32(dst), "copy_tokens": _int32(tokens)}


def _exact_copy(s):
    whole = [s["case"]["page"]] * s["case"]["pairs"]
    out = {}
    for name in ("k", "v"):
        before = s[name].double()
        after = before.clone()
        for a, b, n in zip(s["src"].tolist(), s["dst"].tolist(), s["tokens"].tolist() if s["tokens"] is not None else whole):
            after[:, b, :n] = before[:, a, :n]
        out[name] = after
    return out


def _exact_shared(s):
    c = s["case"]
    h, kv, d, p = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    bytes_ = (lambda x: x.view(torch.uint8)) if c["cache"] == "fp8" else (lambda x: x)
    for r, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        pages = s["table"][r, :_ceil(length, p)].long()                # by the sequence's own row, common pages and all
        keys, vals = (bytes_(x)[pages].view(x.dtype).reshape(-1, kv, d)[:length].double().transpose(0, 1) * y
                      for x, y in ((s["k"], s["scales"][0]), (s["v"], s["scales"][1])))
        for i in range(starts[r], starts[r + 1]):
            seen = length - (starts[r + 1] - i) + 1
            z = torch.bmm(s["q"][i].double().view(kv, h // kv, d), keys[:, :seen].transpose(1, 2).contiguous()) * s["scale"]
            lse[i] = torch.logsumexp(z, -1).reshape(h)
            out[i] = torch.bmm(torch.softmax(z, -1), vals[:, :seen].contiguous()).reshape(h * d)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"select": _exact_select, "fork": _exact_fork, "copy": _exact_copy, "shared": _exact_shared}[case["op"]](s)
