"""The serving operators that surround the LoRA projections of an attention layer, as measured cases.

Three operators, in the order a decode step uses them after the packed q/k/v projection:

  plan    block table, slot map and positions of a step, built on the GPU from request lengths
  append  rotary positions on the packed q/k/v rows, keys and values written into the paged cache
  attend  attention of the new tokens over the paged cache

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
        # eight chats, one new token each: the smallest step, bound by latency
        {"name": "plan-decode-8", "op": "plan", "seqs": 8, "past_lo": 40, "past_hi": 2000, "new_lo": 1, "new_hi": 1,
         "ended": 0, "page": 16, "short": 0},
        # a busy server's decode step: 1024 requests, some of which have just ended and give their pages back
        {"name": "plan-decode-1024", "op": "plan", "seqs": 1024, "past_lo": 17, "past_hi": 8191, "new_lo": 1, "new_hi": 1,
         "ended": 37, "page": 16, "short": 0},
        # prompts and decode tokens in one step, with too few free pages for the last requests
        {"name": "plan-mixed-200", "op": "plan", "seqs": 200, "past_lo": 1, "past_hi": 3000, "new_lo": 1, "new_hi": 1500,
         "ended": 11, "page": 32, "short": 40},
        # 64 decode tokens of a layer with 32 query and 8 key/value heads of 128
        {"name": "append-decode-64", "op": "append", "tokens": 64, "new": 1, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "pos_hi": 4096, "factor": 1.0, "cache": "bf16", "page": 16, "order": "token"},
        # sixteen prompts of 276 or 277 tokens each (a prefill batch of 4425 tokens)
        {"name": "append-prefill-4425", "op": "append", "tokens": 4425, "new": 277, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "pos_hi": 512, "factor": 1.0, "cache": "bf16", "page": 16, "order": "token"},
        # far positions, frequencies scaled for a long context, half of the head rotated, an 8-bit cache
        {"name": "append-far-fp8-256", "op": "append", "tokens": 256, "new": 4, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 64, "interleaved": True, "pos_hi": 1000000, "factor": 8.0, "cache": "fp8", "page": 64, "order": "head"},
        # float32 activations, heads of 80 with 20 rotated pairs, an odd token count
        {"name": "append-f32-999", "op": "append", "tokens": 999, "new": 333, "q_heads": 12, "kv_heads": 4, "dim": 80,
         "rot": 40, "interleaved": False, "pos_hi": 8192, "factor": 1.0, "cache": "f32", "page": 32, "order": "token"},
        # one chat, one token: latency
        {"name": "attend-1x777", "op": "attend", "seqs": 1, "len_lo": 777, "len_hi": 777, "new": 1, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16, "order": "token", "window": 0, "idle": 0},
        # 64 chats of 128 to 4096 tokens
        {"name": "attend-64x4096", "op": "attend", "seqs": 64, "len_lo": 128, "len_hi": 4096, "new": 1, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16, "order": "token", "window": 0, "idle": 1},
        # one long document
        {"name": "attend-1x131071", "op": "attend", "seqs": 1, "len_lo": 131071, "len_hi": 131071, "new": 1, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 64, "order": "head", "window": 0, "idle": 0},
        # verification of three drafted tokens over an 8-bit cache
        {"name": "attend-draft-fp8-32x8192", "op": "attend", "seqs": 32, "len_lo": 1000, "len_hi": 8192, "new": 4,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "cache": "fp8", "page": 64, "order": "token", "window": 0, "idle": 0},
        # a full server: 256 chats of about 2000 to 4000 tokens, 4 GB of cache
        {"name": "attend-256x4000", "op": "attend", "seqs": 256, "len_lo": 2000, "len_hi": 4000, "new": 1, "q_heads": 32,
         "kv_heads": 8, "dim": 128, "cache": "bf16", "page": 16, "order": "token", "window": 0, "idle": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend"])
    if op == "plan":
        seqs = _log_int(rng, 1, 1024)
        past_hi = _log_int(rng, 1, 8192)
        new_hi = rng.choice([1, 1, rng.randint(2, 8), min(2000, 65536 // seqs)])
        return {"op": op, "seqs": seqs, "past_lo": rng.randint(0, past_hi), "past_hi": past_hi, "new_lo": 1,
                "new_hi": max(1, new_hi), "ended": rng.randint(0, seqs // 4), "page": rng.choice([16, 32, 64, 128]),
                "short": rng.choice([0, 0, rng.randint(1, 50)])}
    kv_heads = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    cache = rng.choice(["bf16", "bf16", "fp8", "f32"])
    page, order = rng.choice([16, 32, 64, 128]), rng.choice(["token", "head"])
    if op == "append":
        group = rng.randint(1, 8)
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(4, dim // 2)
        most = min(8192, (1 << 25) // (kv_heads * (group + 2) * dim * (2 if cache == "f32" else 1)))
        tokens = _log_int(rng, 1, most)
        return {"op": op, "tokens": tokens, "new": rng.choice([1, 4, rng.randint(1, tokens)]), "q_heads": kv_heads * group,
                "kv_heads": kv_heads, "dim": dim, "rot": rot, "interleaved": rng.random() < 0.5,
                "pos_hi": _log_int(rng, tokens + 1, 2000000), "factor": rng.choice([1.0, 4.0, 8.0]), "cache": cache,
                "page": page, "order": order}
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
    row = 2 * kv_heads * dim * SIZES[cache]              # bytes of one token in the cache
    seqs = _log_int(rng, 1, 256)
    len_hi = _log_int(rng, 8, max(8, min(131072, 2_000_000_000 // (row * seqs))))
    return {"op": op, "seqs": seqs, "len_lo": _log_int(rng, 8, len_hi), "len_hi": len_hi, "new": rng.choice([1, 1, 1, 2, 5, 8]),
            "q_heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page, "order": order,
            "window": rng.choice([0, 0, _log_int(rng, 16, 8192)]), "idle": rng.choice([0, 1]) if seqs > 1 else 0}


# ------------------------------------------------------------------------------------ sizes that follow from a case
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _ceil(a, b):
    return -(-a // b)


def _plan_sizes(case):
    """(past, new) of every request: prompts of all lengths in the range, the last `ended` requests over (-1)."""
    n, e = case["seqs"], case["ended"]
    past, new = _spread(case["past_lo"], case["past_hi"], n), _spread(case["new_lo"], case["new_hi"], n - e)
    return past, [new[(i * 7) % len(new)] for i in range(n - e)] + [-1] * e


def _append_lens(case):
    t, new = case["tokens"], case["new"]
    return [new] * (t // new) + ([t % new] if t % new else [])


def _attend_lens(case):
    """(lengths, new tokens) of every sequence; the first `idle` of them have nothing in the cache."""
    lens = _spread(case["len_lo"], case["len_hi"], case["seqs"])
    new = [min(case["new"], x) for x in lens]
    return [0 if i < case["idle"] else x for i, x in enumerate(lens)], new


def _seen(length, new, window):
    """Cached tokens that the `new` last tokens see."""
    return length if not window else min(length, window + new - 1)


def _act(case):
    return "f32" if case["cache"] == "f32" else "bf16"


def work(case):
    if case["op"] == "plan":
        past, new = _plan_sizes(case)
        p, live = case["page"], [(a, b) for a, b in zip(past, new) if b >= 0]
        tokens = sum(b for _, b in live)
        fresh = sum(_ceil(a + b, p) - _ceil(a, p) for a, b in live)
        back = sum(_ceil(a, p) for a, b in zip(past, new) if b < 0)
        # lengths in, lengths and starts out, position and slot of each token (and the page it lies in), moved pages
        return {"bytes": 16 * len(past) + 8 * tokens + 8 * fresh + 8 * back, "flops": 4 * tokens}
    if case["op"] == "append":
        t, q, kv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        act, cell = SIZES[_act(case)], SIZES[case["cache"]]
        return {"bytes": t * ((2 * q + 2 * kv) * d * act + 2 * kv * d * cell + 8), "flops": 3 * t * (q + kv) * case["rot"]}
    lens, new = _attend_lens(case)
    seen = sum(_seen(a, b, case["window"]) for a, b in zip(lens, new))
    pairs = sum(_seen(a, b, case["window"]) * b for a, b in zip(lens, new))
    d, act = case["dim"], SIZES[_act(case)]
    return {"bytes": 2 * seen * case["kv_heads"] * d * SIZES[case["cache"]] + 2 * sum(new) * case["q_heads"] * d * act
            + 4 * sum(_ceil(a, case["page"]) for a in lens) + 8 * len(lens),
            "flops": 4 * pairs * case["q_heads"] * d}


# ------------------------------------------------------------------------------------ inputs
def _frequencies(case):
    """Rotary frequencies (radians a position): base^(-2i/rot); with a factor, those whose wavelength passes 8192
    positions divided by it, those under 2048 kept, and the ones between blended by original_len / wavelength."""
    rot = case["rot"]
    f = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["factor"] == 1.0:
        return f
    blend = [min(1.0, max(0.0, (8192.0 * x / (2.0 * math.pi) - 1.0) / 3.0)) for x in f]
    return [x * (b + (1.0 - b) / case["factor"]) for x, b in zip(f, blend)]


def _int32(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _cache(case, pages, gen):
    """Keys or values [pages, page, heads, dim] in the order of the case."""
    kv, d, p = case["kv_heads"], case["dim"], case["page"]
    shape = (pages, p, kv, d) if case["order"] == "token" else (pages, kv, p, d)
    x = torch.empty(shape, dtype=DTYPES[case["cache"]], device="cuda")
    step = max(1, (1 << 28) // (p * kv * d))
    for i in range(0, pages, step):
        part = x[i:i + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return x if case["order"] == "token" else x.transpose(1, 2)


def _inputs(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "plan":
        past, new = _plan_sizes(case)
        order = list(range(len(past)))
        rng.shuffle(order)
        past, new = [past[i] for i in order], [new[i] for i in order]
        p = case["page"]
        held = sum(_ceil(a, p) for a in past)
        need = sum(_ceil(a + max(b, 0), p) - _ceil(a, p) for a, b in zip(past, new))
        free = max(0, need - case["short"]) if case["short"] else need + 3 + need // 4
        pages = held + free
        ids = np.random.default_rng(seed).permutation(pages).astype(np.int32)
        width = max(_ceil(a + max(b, 0), p) for a, b in zip(past, new)) + 2
        table = np.full((len(past), width), -1, dtype=np.int32)
        at = 0
        for i, a in enumerate(past):
            n = _ceil(a, p)
            table[i, :n] = ids[at:at + n]
            at += n
        ring = np.full(pages, -1, dtype=np.int32)
        head = rng.randrange(pages)
        ring[(head + np.arange(free)) % pages] = ids[at:]
        s.update(past=_int32(past), new=_int32(new), tokens=sum(b for b in new if b > 0), pages=pages,
                 table=torch.from_numpy(table).cuda(), ring=torch.from_numpy(ring).cuda(),
                 cursor=_int32([head, free, 0, 0]), cursor_out=_int32([0, 0, 0, 0]))
        return s
    if case["op"] == "append":
        t, p = case["tokens"], case["page"]
        lens = _append_lens(case)
        starts = [rng.randint(0, max(0, case["pos_hi"] - n)) for n in lens]
        spare = [_ceil(n + p - 1, p) for n in lens]                      # the most pages that the new tokens touch
        pages = sum(spare) + 5
        ids = list(range(pages))
        rng.shuffle(ids)
        positions, slots, at = [], [], 0
        for a, n, m in zip(starts, lens, spare):
            mine = np.array(ids[at:at + m])
            at += m
            x = np.arange(a, a + n)
            positions.append(x)
            slots.append(mine[(x - a // p * p) // p] * p + x % p)
        width = (case["q_heads"] + 2 * case["kv_heads"]) * case["dim"]
        act = DTYPES[_act(case)]
        scales = (0.75, 1.25) if case["cache"] == "fp8" else (1.0, 1.0)
        s.update(qkv=torch.randn((t, width), generator=gen, device="cuda").to(act),
                 q_out=torch.zeros((t, case["q_heads"] * case["dim"]), dtype=act, device="cuda"),
                 k=_cache(case, pages, gen), v=_cache(case, pages, gen), scales=scales,
                 positions=torch.from_numpy(np.concatenate(positions).astype(np.int32)).cuda(),
                 slots=torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda(),
                 freqs=_frequencies(case), amplitude=1.0 if case["factor"] == 1.0 else 1.125)
        s["freqs_gpu"] = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
        return s
    lens, new = _attend_lens(case)
    order = list(range(len(lens)))
    rng.shuffle(order)
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    p = case["page"]
    need = [_ceil(a, p) for a in lens]
    pages = sum(need) + 3
    ids = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(1, max(need)) + 1), -1, dtype=np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    act = DTYPES[_act(case)]
    t = sum(new)
    scales = (0.75, 1.25) if case["cache"] == "fp8" else (1.0, 1.0)
    s.update(q=torch.randn((t, case["q_heads"] * case["dim"]), generator=gen, device="cuda").mul_(1.5).to(act),
             k=_cache(case, pages, gen), v=_cache(case, pages, gen), scales=scales, table=torch.from_numpy(table).cuda(),
             lens=_int32(lens), starts=_int32([0] + np.cumsum(new).tolist()), longest=max(1, max(lens)), most=max(new),
             out=torch.zeros((t, case["q_heads"] * case["dim"]), dtype=act, device="cuda"),
             lse=torch.zeros((t, case["q_heads"]), dtype=torch.float32, device="cuda"),
             scale=1.0 / math.sqrt(case["dim"]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import rank_adapter_gemm_build_amd as rx
        if case["op"] == "plan":
            s["plan"] = rx.PagePlan(0, case["seqs"], max(1, s["tokens"]))
        else:
            s["kv"] = rx.KVCache(s["k"], s["v"], *s["scales"])
            if case["op"] == "append":
                s["rotary"] = rx.Rotary(0, case["rot"], s["freqs"], interleaved=case["interleaved"], amplitude=s["amplitude"])
            else:
                s["attention"] = rx.Attention(0, case["seqs"], s["q"].shape[0], case["q_heads"], case["kv_heads"], case["dim"])
    return s


# ------------------------------------------------------------------------------------ plain forms
def _plain_plan(s):
    past, new, table, ring, p = s["past"].long(), s["new"].long(), s["table"], s["ring"], s["case"]["page"]
    head, free, pages = s["cursor"][0].long(), s["cursor"][1].long(), s["pages"]
    count = new.clamp(min=0)
    ends = count.cumsum(0)
    start = ends - count
    have = (past + p - 1) // p
    need = torch.where(new >= 0, (past + count + p - 1) // p - have, 0)
    last = need.cumsum(0)
    first = last - need
    granted = (new >= 0) & ((need == 0) | (last <= free))
    taken = torch.where(granted, last, 0).max()
    # tokens
    t = torch.arange(s["tokens"], device=past.device)
    r = torch.searchsorted(ends, t, right=True)
    pos = past[r] + t - start[r]
    # new pages into the table
    col = torch.arange(table.shape[1], device=past.device)
    fresh = (granted & (need > 0))[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    rank = first[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, ring[(head + rank.clamp(min=0)) % pages], table))
    slots = torch.where(granted[r], table[r, (pos // p).clamp(max=table.shape[1] - 1)].long() * p + pos % p, -1)
    # pages of ended requests back to the ring's end
    back = torch.where(new < 0, have, 0)
    before = back.cumsum(0) - back
    gone = col < back[:, None]
    place = (head + free + before[:, None] + col) % pages
    ring[place[gone]] = table[gone]
    s["cursor_out"][:2] = torch.stack([(head + taken) % pages, free - taken + back.sum()]).int()
    lens = torch.where(granted, past + count, 0)
    return {"seq_lens": lens.int(), "query_start": torch.cat([ends.new_zeros(1), ends]).int(), "positions": pos.int(),
            "slots": slots.int(), "table": table, "free_pages": ring, "cursor": s["cursor_out"]}


def _turn(x, cos, sin, rot, interleaved):
    """The first `rot` values of each head turned: x [t, heads, dim], cos and sin [t, rot / 2]."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], dim=-1).flatten(-2) if interleaved else torch.cat([u, w], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    c = s["case"]
    t, h, kv, d, p = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    x = s["qkv"].float().view(t, h + 2 * kv, d)
    angle = s["positions"].double()[:, None] * s["freqs_gpu"]
    cos, sin = (angle.cos() * s["amplitude"]).float(), (angle.sin() * s["amplitude"]).float()
    y = _turn(x[:, :h + kv], cos, sin, c["rot"], c["interleaved"])
    s["q_out"].copy_(y[:, :h].reshape(t, h * d))
    page, at = s["slots"].long() // p, s["slots"].long() % p
    k, v = y[:, h:], x[:, h + kv:]
    if c["cache"] == "fp8":
        k, v = (k / s["scales"][0]).clamp(-448, 448), (v / s["scales"][1]).clamp(-448, 448)
        s["k"].view(torch.uint8)[page, at] = k.to(E4M3).view(torch.uint8)
        s["v"].view(torch.uint8)[page, at] = v.to(E4M3).view(torch.uint8)
    else:
        s["k"][page, at] = k.to(s["k"].dtype)
        s["v"][page, at] = v.to(s["v"].dtype)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["case"]
    h, kv, d, p = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    n, m, g, longest = len(s["lens"]), s["most"], h // kv, s["longest"]
    lens, starts = s["lens"].long(), s["starts"].long()
    j = torch.arange(longest, device="cuda")
    page = s["table"].long()[:, j // p].clamp(min=0)                                  # [n, longest]
    bytes_ = (lambda x: x.view(torch.uint8)) if c["cache"] == "fp8" else (lambda x: x)
    keys = bytes_(s["k"])[page, j % p].view(s["k"].dtype).float() * s["scales"][0]       # [n, longest, kv, d]
    vals = bytes_(s["v"])[page, j % p].view(s["v"].dtype).float() * s["scales"][1]
    count = starts[1:] - starts[:-1]
    i = torch.arange(m, device="cuda")
    there = i < count[:, None]
    row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[row].view(n, m, kv, g, d).permute(0, 2, 1, 3, 4).reshape(n, kv, m * g, d)
    score = torch.matmul(q, keys.permute(0, 2, 3, 1)).view(n, kv, m, g, longest) * s["scale"]
    pos = lens[:, None] - count[:, None] + i
    see = (j <= pos[:, :, None]) & (j < lens[:, None, None])
    if c["window"]:
        see = see & (j > pos[:, :, None] - c["window"])
    score = score.masked_fill(~see[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul((e / total.clamp(min=1e-38)).view(n, kv, m * g, longest), vals.permute(0, 2, 1, 3))
    o = o.view(n, kv, m, g, d).permute(0, 2, 1, 3, 4).reshape(n, m, h * d)
    lse = (top + total.log()).view(n, kv, m, g).permute(0, 2, 1, 3).reshape(n, m, h)
    s["out"].copy_(o[there])
    s["lse"].copy_(lse[there])
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attend": _plain_attend}[op](s)
    import rank_adapter_gemm_build_amd as rx
    if op == "plan":
        plan = s["plan"]
        rx.page_plan(plan, s["past"], s["new"], s["tokens"], s["ring"], s["cursor"], s["table"], s["case"]["page"],
                     cursor_out=s["cursor_out"])
        n, t = s["case"]["seqs"], s["tokens"]
        return {"seq_lens": plan.seq_lens[:n], "query_start": plan.query_start[:n + 1], "positions": plan.positions[:t],
                "slots": plan.slots[:t], "table": s["table"], "free_pages": s["ring"], "cursor": s["cursor_out"]}
    if op == "append":
        rx.rotary_append(s["rotary"], s["qkv"], s["case"]["q_heads"], s["positions"], s["slots"], s["q_out"], s["kv"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    rx.paged_attention(s["attention"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], s["out"], scale=s["scale"],
                       window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------ the definitions, in 64 bits
def _exact_plan(s):
    case, p, pages = s["case"], s["case"]["page"], s["pages"]
    past, new = s["past"].tolist(), s["new"].tolist()
    table, ring = s["table"].cpu().numpy().copy(), s["ring"].cpu().numpy().copy()
    head, free = s["cursor"].tolist()[:2]
    lens, starts, positions, slots = [], [0], [], []
    asked = taken = 0
    for r in range(case["seqs"]):
        n = max(new[r], 0)
        starts.append(starts[-1] + n)
        have, all_ = _ceil(past[r], p), _ceil(past[r] + n, p)
        asked += all_ - have if new[r] >= 0 else 0
        fits = new[r] >= 0 and (all_ == have or asked <= free)
        if fits and all_ > have:
            for e in range(all_ - have):
                table[r, have + e] = ring[(head + taken + e) % pages]
            taken += all_ - have
        lens.append(past[r] + n if fits else 0)
        x = np.arange(past[r], past[r] + n)
        positions.append(x)
        slots.append(table[r, x // p].astype(np.int64) * p + x % p if fits else np.full(n, -1))
    tail = head + free
    for r in range(case["seqs"]):
        if new[r] < 0:
            for e in range(_ceil(past[r], p)):
                ring[tail % pages] = table[r, e]
                tail += 1
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()  # noqa: E731
    return {"seq_lens": i32(lens), "query_start": i32(starts), "positions": i32(np.concatenate(positions)),
            "slots": i32(np.concatenate(slots)), "table": i32(table), "free_pages": i32(ring),
            "cursor": i32([(head + taken) % pages, tail - head - taken, 0, 0])}


def _exact_append(s):
    c = s["case"]
    t, h, kv, d, rot, p = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["rot"], c["page"]
    x = s["qkv"].double().view(t, h + 2 * kv, d)
    angle = torch.outer(s["positions"].double(), torch.tensor(s["freqs"], dtype=torch.float64, device="cuda"))
    wave = torch.polar(torch.full_like(angle, s["amplitude"]), angle)                 # pairs as complex numbers
    first = torch.arange(rot // 2, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else rot // 2)
    z = torch.complex(x[:, :h + kv][..., first], x[:, :h + kv][..., second]) * wave[:, None]
    y = x[:, :h + kv].clone()
    y[..., first], y[..., second] = z.real, z.imag
    k, v = s["k"].double(), s["v"].double()
    page, at = s["slots"].long() // p, s["slots"].long() % p
    k[page, at], v[page, at] = y[:, h:] / s["scales"][0], x[:, h + kv:] / s["scales"][1]
    if c["cache"] == "fp8":
        k, v = k.clamp(-448, 448), v.clamp(-448, 448)
    return {"q": y[:, :h].reshape(t, h * d), "k": k, "v": v}


def _exact_attend(s):
    c = s["case"]
    h, kv, d, p = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    for r, length in enumerate(s["lens"].tolist()):
        a, b = starts[r], starts[r + 1]
        if length == 0:
            continue
        pages = s["table"][r, :_ceil(length, p)].long()
        bytes_ = (lambda x: x.view(torch.uint8)[pages].view(E4M3)) if c["cache"] == "fp8" else (lambda x: x[pages])
        keys = bytes_(s["k"]).reshape(-1, kv, d)[:length].double() * s["scales"][0]
        vals = bytes_(s["v"]).reshape(-1, kv, d)[:length].double() * s["scales"][1]
        for i in range(a, b):
            pos = length - (b - i)
            lo = max(0, pos - c["window"] + 1) if c["window"] else 0
            if pos < lo:
                continue
            q = s["q"][i].double().view(kv, h // kv, d)
            z = torch.einsum("kgd,jkd->kgj", q, keys[lo:pos + 1]) * s["scale"]
            lse[i] = torch.logsumexp(z, -1).reshape(h)
            out[i] = torch.einsum("kgj,jkd->kgd", torch.softmax(z, -1), vals[lo:pos + 1]).reshape(h * d)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
