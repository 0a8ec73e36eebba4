"""Beam search on a LoRA server over a paged cache, step by step as a server runs it.

A prompt step, in which each request's first beam alone has tokens, then decode steps replayed from one captured graph:

    page plan -> per layer: packed q/k/v projection + its LoRA correction -> rotary append -> shared attention ->
    o projection -> logits -> beam selection -> page fork -> page copy

The beams of a request share its prompt's pages, and every prefix of tokens that they have in common; the shared attention reads
the prompt once for all of them.  Beams that end keep their place in the ranking and give back their pages.
Every step's logits are compared with a dense recomputation of each beam's whole history, and the choice with a plain one
over the same logits.  python examples/beam_search.py"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import rank_adapter_gemm_build_amd as rx  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE, LAYERS, VOCAB, RANK = 256, 8, 2, 64, 16, 2, 500, 8
WIDTH, PROMPTS, SLOT_OF, END = 4, [37, 64, 5], [0, 1, -1], 7
REQUESTS, ROWS = len(PROMPTS), WIDTH * len(PROMPTS)
MAX_LEN, PAGES = 128, 60
QKV = [HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM]


class Model:
    """Weights, adapters of the q/k/v projections, and the objects a server keeps."""

    def __init__(self, seed: int):
        rng = np.random.default_rng(seed)

        def weight(*shape, gain=1.0):
            return torch.from_numpy((rng.normal(size=shape) * gain / np.sqrt(shape[-1])).astype(np.float32)).bfloat16().cuda()
        self.embed = weight(VOCAB, HIDDEN, gain=np.sqrt(HIDDEN))
        self.head, self.bias = weight(VOCAB, HIDDEN), torch.zeros(VOCAB, dtype=torch.bfloat16, device="cuda")
        self.bias[END] = 4.0                           # so that some beams end
        self.w_qkv, self.w_o = [weight(sum(QKV), HIDDEN) for _ in range(LAYERS)], [weight(HIDDEN, HEADS * DIM) for _ in range(LAYERS)]
        slots, tokens = max(SLOT_OF) + 1, max(sum(PROMPTS), ROWS)
        self.pools = [rx.Pool(0, slots, RANK, HIDDEN, QKV, rx.LORA_BF16, tokens) for _ in range(LAYERS)]
        self.adapters = [[[(weight(RANK, HIDDEN), weight(d, RANK, gain=2.0)) for d in QKV] for _ in range(slots)] for _ in range(LAYERS)]
        for pool, of_layer in zip(self.pools, self.adapters):
            for s, pairs in enumerate(of_layer):
                pool.register(s, [a for a, _ in pairs], [b for _, b in pairs], 0.5 * RANK, RANK)
        self.freqs = rx.rotary_frequencies(DIM, 10000.0)
        self.rotary, self.routing = rx.Rotary(0, DIM, self.freqs), rx.Routing(0, tokens, slots)
        self.attention = rx.SharedAttention(0, ROWS, tokens, HEADS, KV_HEADS, DIM)
        self.beams = rx.Beams(0, REQUESTS, WIDTH, VOCAB)
        self.layers = rx.KVLayers(rx.KVCache(*(torch.zeros(PAGES, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in "kv"))
                                  for _ in range(LAYERS))

    def dense(self, tokens, slot):
        """Logits after a row's whole history, in float32."""
        n = len(tokens)
        x = self.embed[torch.tensor(tokens, device="cuda")].float()
        angle = (torch.arange(n, device="cuda").double()[:, None] * torch.tensor(self.freqs, dtype=torch.float64, device="cuda")).float()
        c, s, half = angle.cos()[:, None], angle.sin()[:, None], DIM // 2
        for layer in range(LAYERS):
            h = x @ self.w_qkv[layer].float().t()
            if slot >= 0:
                h = h + torch.cat([0.5 * (x @ a.float().t()) @ b.float().t() for a, b in self.adapters[layer][slot]], 1)
            h = h.view(n, HEADS + 2 * KV_HEADS, DIM)
            a, b = h[..., :half], h[..., half:]
            turned = torch.cat([a * c - b * s, a * s + b * c], -1)
            q, k, v = turned[:, :HEADS], turned[:, HEADS:HEADS + KV_HEADS], h[:, HEADS + KV_HEADS:]
            k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1).contiguous() for t in (k, v))
            score = torch.bmm(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) / DIM ** 0.5
            score = score.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -float("inf"))
            x = x + torch.bmm(score.softmax(-1), v).transpose(0, 1).reshape(n, HEADS * DIM) @ self.w_o[layer].float().t()
        return x[-1] @ self.head.float().t() + self.bias.float()


class Search:
    """What a server keeps of the requests in flight: all of it on the device, at fixed addresses."""

    def __init__(self, model: Model):
        self.model = model
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((ROWS, MAX_LEN // PAGE), -1, **i32)
        self.ring, self.cursor, self.shares = torch.arange(PAGES, **i32), torch.tensor([0, PAGES, 0, 0], **i32), torch.zeros(PAGES, **i32)
        tokens = max(sum(PROMPTS), ROWS)
        self.plan, self.fork = rx.PagePlan(0, ROWS, tokens), rx.ForkPlan(0, ROWS, PAGES)
        self.lens, self.new, self.ended = (torch.zeros(ROWS, **i32) for _ in range(3))
        self.parents, self.heirs, self.tokens = (torch.full((ROWS,), -1, **i32) for _ in range(3))
        self.before, self.scores = torch.zeros(ROWS, device="cuda"), torch.full((ROWS,), -float("inf"), device="cuda")
        self.scores[::WIDTH] = 0.0                                             # one beam a request to begin with
        self.group_start, self.common = torch.arange(REQUESTS + 1, **i32) * WIDTH, torch.tensor(PROMPTS, **i32)
        self.slot_of_row = torch.tensor(SLOT_OF, **i32).repeat_interleave(WIDTH)
        self.none, self.end = torch.full((ROWS,), -1, **i32), torch.full((ROWS,), END, **i32)
        self.logits = torch.zeros(ROWS, VOCAB, dtype=torch.bfloat16, device="cuda")

    def buffers(self, T):
        def rows(*shape, dtype=torch.bfloat16):
            return torch.zeros(T, *shape, dtype=dtype, device="cuda")
        return dict(x=rows(HIDDEN), qkv=rows(sum(QKV)), q=rows(HEADS * DIM), attended=rows(HEADS * DIM), y=rows(HIDDEN),
                    slots=rows(dtype=torch.int32))

    def forward(self, b):
        """The rows' new tokens (b["x"], their adapters b["slots"]) through the layers, and the logits of each row's last one."""
        m, plan, T = self.model, self.plan, b["x"].shape[0]
        for layer, cache in enumerate(m.layers.caches):
            torch.matmul(b["x"], m.w_qkv[layer].t(), out=b["qkv"])
            rx.route_linear(m.pools[layer], m.routing, b["slots"], b["x"], b["qkv"])
            rx.rotary_append(m.rotary, b["qkv"], HEADS, plan.positions[:T], plan.slots[:T], b["q"], cache)
            rx.shared_attention(m.attention, b["q"], cache, self.table, plan.seq_lens[:ROWS], plan.query_start[:ROWS + 1], self.group_start,
                                self.common, b["attended"])
            torch.matmul(b["attended"], m.w_o[layer].t(), out=b["y"])
            b["x"].add_(b["y"])
        last = (plan.query_start[1:ROWS + 1] - 1).clamp_(min=0)               # a row without new tokens gets another's: never read
        torch.matmul(b["x"].index_select(0, last), m.head.t(), out=self.logits)
        self.logits.add_(m.bias)

    def choose(self):
        """The best continuations, and the rows that hold them from now on."""
        m = self.model
        self.lens.copy_(self.plan.seq_lens[:ROWS])
        self.before.copy_(self.scores)
        rx.beam_select(m.beams, self.logits, self.scores, self.parents, self.tokens, self.scores, ended=self.ended, end_token=END,
                       ended_out=self.ended)
        self.heirs.copy_(torch.where(self.ended > 0, self.none, self.parents))    # a beam that has ended needs no keys any more
        rx.page_fork(self.fork, self.heirs, self.lens, self.ring, self.cursor, self.shares, self.table, PAGE)
        rx.page_copy(m.layers, self.fork.copy_src, self.fork.copy_dst, self.fork.copy_tokens)

    def prompt(self, prompts):
        b = self.buffers(sum(PROMPTS))
        self.new[::WIDTH] = torch.tensor(PROMPTS, dtype=torch.int32, device="cuda")
        rx.page_plan(self.plan, self.lens, self.new, sum(PROMPTS), self.ring, self.cursor, self.table, PAGE)
        b["x"].copy_(self.model.embed[torch.tensor([t for p in prompts for t in p], device="cuda")])
        b["slots"].copy_(torch.tensor([s for s, p in zip(SLOT_OF, prompts) for _ in p], dtype=torch.int32))
        self.forward(b)
        self.choose()

    def decode(self, b):
        """One token for every beam that goes on."""
        m = self.model
        self.new.copy_((self.heirs >= 0).int())
        rx.page_plan(self.plan, self.lens, self.new, ROWS, self.ring, self.cursor, self.table, PAGE)
        # the plan packs the rows that have a token; place ROWS takes what the others have
        at = torch.where(self.new > 0, self.plan.query_start[:ROWS], torch.full_like(self.new, ROWS)).long()
        b["packed"].fill_(-1).scatter_(0, at, torch.arange(ROWS, device="cuda"))
        row = b["packed"][:ROWS].clamp(min=0)
        b["x"].copy_(m.embed.index_select(0, self.tokens.index_select(0, row).clamp(min=0)))
        b["slots"].copy_(torch.where(b["packed"][:ROWS] >= 0, self.slot_of_row.index_select(0, row), self.none))
        self.forward(b)
        self.choose()


def main(steps: int = 14, seed: int = 0) -> float:
    """Largest error of any step's logits, relative to the dense ones' largest value."""
    model = Model(seed)
    search = Search(model)
    rng = np.random.default_rng(seed)
    prompts = [rng.integers(0, VOCAB, n).tolist() for n in PROMPTS]
    held = [prompts[r // WIDTH] if r % WIDTH == 0 else None for r in range(ROWS)]   # the history that a row's cache has, with its new token
    worst, ended_before = 0.0, [0] * ROWS
    ends = 0

    def check():
        nonlocal worst, held, ended_before, ends
        live = [r for r in range(ROWS) if held[r] is not None and not ended_before[r]]
        for r in live:
            want = model.dense(held[r], SLOT_OF[r // WIDTH])
            worst = max(worst, float((search.logits[r].float() - want).abs().max() / want.abs().max()))
        # the choice, over the same logits in 64 bits
        before, parents, tokens = search.before.tolist(), search.parents.tolist(), search.tokens.tolist()
        scores, ended, heirs = search.scores.tolist(), search.ended.tolist(), search.heirs.tolist()
        logp = torch.log_softmax(search.logits.double(), -1)
        for g in range(REQUESTS):
            found = []
            for r in range(g * WIDTH, (g + 1) * WIDTH):
                if ended_before[r]:
                    found.append((before[r], r, END))
                elif r in live:
                    top = torch.topk(logp[r], WIDTH)
                    found += [(before[r] + p, r, t) for p, t in zip(top.values.tolist(), top.indices.tolist())]
            for i, (s, _, _) in enumerate(sorted(found, reverse=True)[:WIDTH]):
                at = g * WIDTH + i
                assert abs(scores[at] - s) <= 1e-4 + 2.0 ** -22 * abs(s), "a better continuation was passed over"
                p, t = parents[at], tokens[at]
                assert p // WIDTH == g and (ended_before[p] or abs(before[p] + float(logp[p, t]) - scores[at]) <= 1e-4 + 2.0 ** -22 * abs(s))
        # a place without a continuation of its own (ended, or fewer than the width) holds no keys
        held = [held[parents[r]] + [tokens[r]] if heirs[r] >= 0 else None for r in range(ROWS)]
        ends += sum(ended) - sum(ended_before)
        ended_before = ended
        assert search.fork.query()["refused"] == 0 and search.fork.query()["invalid"] == 0 and search.plan.query()["refused"] == 0

    search.prompt(prompts)
    check()
    b = search.buffers(ROWS)
    b["packed"] = torch.zeros(ROWS + 1, dtype=torch.int64, device="cuda")
    search.decode(b)                              # the first one eagerly: library set-up stays out of the graph
    check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        search.decode(b)
    for _ in range(steps):
        graph.replay()
        check()
    assert ends > 0, "some beams were to end"
    # all requests are done: every page comes back
    search.heirs.fill_(-1)
    rx.page_fork(search.fork, search.heirs, search.lens, search.ring, search.cursor, search.shares, search.table, PAGE)
    assert search.fork.query()["free_pages"] == PAGES and not search.shares.any(), "pages lost"
    print(f"beam search ok: {steps + 2} steps of {REQUESTS} requests with {WIDTH} beams, {ends} beams ended, largest error of a logit {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
