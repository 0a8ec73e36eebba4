"""One attention layer of a LoRA server over a paged cache, step by step as a server runs it.

A prompt step (requests with prompts of different lengths), decode steps replayed from one
captured graph, a step in which a request ends and another comes in its pages, steps with too
few pages, whose last request is refused until pages have come back, each:

    page plan -> packed q/k/v projection + its LoRA correction -> rotary append ->
    paged attention -> o projection + its LoRA correction

Every step's output is compared with a dense recomputation from the requests' whole
histories.  python examples/paged_serving.py"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

import rank_adapter_gemm_build_amd as rx  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE, SLOTS, RANK, SCALE = 512, 8, 2, 64, 16, 3, 8, 0.5
REQUESTS, MAX_LEN, PAGES, MAX_TOKENS = 4, 128, 16, 128
QKV = [HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM]


def advance(past, new, seq_lens):
    """The cached lengths after a step, on the device: the plan gives length 0 to ended requests and to refused ones,
    which keep what they have and ask again."""
    past.copy_(torch.where(seq_lens > 0, seq_lens, torch.where(new < 0, 0, past)))


class Layer:
    """Base weights, adapters of the two projections, and the objects a server keeps."""

    def __init__(self, seed: int):
        rng = np.random.default_rng(seed)

        def weight(*shape, gain=1.0):
            return torch.from_numpy((rng.normal(size=shape) * gain / np.sqrt(shape[-1])).astype(np.float32)).bfloat16().cuda()
        self.w_qkv, self.w_o = weight(sum(QKV), HIDDEN), weight(HIDDEN, HEADS * DIM)
        self.qkv_pool = rx.Pool(0, SLOTS, RANK, HIDDEN, QKV, rx.LORA_BF16, MAX_TOKENS)
        self.o_pool = rx.Pool(0, SLOTS, RANK, HEADS * DIM, [HIDDEN], rx.LORA_BF16, MAX_TOKENS)
        self.adapters = []
        for s in range(SLOTS):
            qkv = [(weight(RANK, HIDDEN), weight(d, RANK, gain=2.0)) for d in QKV]
            o = [(weight(RANK, HEADS * DIM), weight(HIDDEN, RANK, gain=2.0))]
            for pool, pairs in ((self.qkv_pool, qkv), (self.o_pool, o)):
                pool.register(s, [a for a, _ in pairs], [b for _, b in pairs], SCALE * RANK, RANK)
            self.adapters.append((qkv, o))
        self.freqs = rx.rotary_frequencies(DIM, 10000.0, "wavelength", factor=4.0, original_len=64, low=1.0, high=4.0)
        self.rotary = rx.Rotary(0, DIM, self.freqs)
        self.attention = rx.Attention(0, REQUESTS, MAX_TOKENS, HEADS, KV_HEADS, DIM)
        self.routing = rx.Routing(0, MAX_TOKENS, SLOTS)
        self.cache = rx.KVCache(*(torch.zeros(PAGES, PAGE, KV_HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in "kv"))

    def step(self, plan, x, slot_ids, qkv, q, attended, y):
        """y = the layer's output for the step's rows x; the plan of the step is made."""
        T, R = x.shape[0], REQUESTS
        torch.matmul(x, self.w_qkv.t(), out=qkv)
        rx.route_linear(self.qkv_pool, self.routing, slot_ids, x, qkv)
        rx.rotary_append(self.rotary, qkv, HEADS, plan.positions[:T], plan.slots[:T], q, self.cache)
        rx.paged_attention(self.attention, q, self.cache, self.table, plan.seq_lens[:R], plan.query_start[:R + 1], attended)
        torch.matmul(attended, self.w_o.t(), out=y)
        rx.linear(self.o_pool, self.routing, attended, y)

    def dense(self, rows, slot):
        """The layer over a request's whole history (rows [n, HIDDEN]), in float32."""
        def project(x, w, pairs):
            delta = [SCALE * (x @ a.float().t()) @ b.float().t() for a, b in pairs] if slot >= 0 else [0.0]
            return x @ w.float().t() + (torch.cat(delta, 1) if slot >= 0 else 0.0)
        qkv_pairs, o_pairs = self.adapters[slot] if slot >= 0 else ([], [])
        n = rows.shape[0]
        x = project(rows.float(), self.w_qkv, qkv_pairs).view(n, HEADS + 2 * KV_HEADS, DIM)
        angle = (torch.arange(n, device="cuda").double()[:, None] * torch.tensor(self.freqs, dtype=torch.float64, device="cuda")).float()
        c, s, half = angle.cos()[:, None], angle.sin()[:, None], DIM // 2
        a, b = x[..., :half], x[..., half:]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
        q, k, v = turned[:, :HEADS], turned[:, HEADS:HEADS + KV_HEADS], x[:, HEADS + KV_HEADS:]
        k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1).transpose(0, 1).contiguous() for t in (k, v))
        score = torch.bmm(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) / DIM ** 0.5
        score = score.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), -float("inf"))
        out = torch.bmm(score.softmax(-1), v).transpose(0, 1).reshape(n, HEADS * DIM)
        return project(out, self.w_o, o_pairs)


def main(decode_steps: int = 6, seed: int = 0) -> float:
    """Largest error of any step, relative to the dense output's largest value."""
    torch.manual_seed(seed)
    layer = Layer(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    layer.table = torch.full((REQUESTS, MAX_LEN // PAGE), -1, **i32)
    ring, cursor = torch.arange(PAGES, **i32), torch.tensor([0, PAGES, 0, 0], **i32)
    plan = rx.PagePlan(0, REQUESTS, MAX_TOKENS)
    past, new = torch.zeros(REQUESTS, **i32), torch.zeros(REQUESTS, **i32)
    slots_of = [0, 1, -1, 2]                      # the adapter of each request (-1: none)
    history = [torch.zeros(0, HIDDEN, dtype=torch.bfloat16, device="cuda") for _ in range(REQUESTS)]
    worst, refusals = 0.0, 0

    def buffers(T):
        def rows(width):
            return torch.zeros(T, width, dtype=torch.bfloat16, device="cuda")
        return rows(HIDDEN), rows(sum(QKV)), rows(HEADS * DIM), rows(HEADS * DIM), rows(HIDDEN)

    def ids_of(counts):
        return torch.tensor([s for s, n in zip(slots_of, counts) for _ in range(max(n, 0))], **i32)

    def check(x, y, counts):
        nonlocal worst, refusals
        granted = plan.seq_lens[:REQUESTS].tolist()
        refusals += plan.query()["refused"]
        at = 0
        for r, n in enumerate(counts):
            if n <= 0:
                continue
            if not granted[r]:                    # nothing of it was stored: its tokens come again
                assert not y[at:at + n].any()
                at += n
                continue
            history[r] = torch.cat([history[r], x[at:at + n]])
            want = layer.dense(history[r], slots_of[r])[-n:]
            worst = max(worst, float((y[at:at + n].float() - want).abs().max() / want.abs().max()))
            at += n

    def eager_step(counts):
        """counts[r]: new tokens of request r, -1 where it has ended"""
        T = sum(max(n, 0) for n in counts)
        x, qkv, q, attended, y = buffers(T)
        x.normal_()
        new.copy_(torch.tensor(counts, **i32))
        rx.page_plan(plan, past, new, T, ring, cursor, layer.table, PAGE)
        layer.step(plan, x, ids_of(counts), qkv, q, attended, y)
        check(x, y, counts)
        advance(past, new, plan.seq_lens[:REQUESTS])

    eager_step([37, 16, 1, 50])                   # prompts
    # decode: one token a request, the whole step in a graph
    x, qkv, q, attended, y = buffers(REQUESTS)
    ids = ids_of([1] * REQUESTS)
    new.fill_(1)

    def decode():
        rx.page_plan(plan, past, new, REQUESTS, ring, cursor, layer.table, PAGE)
        layer.step(plan, x, ids, qkv, q, attended, y)
        advance(past, new, plan.seq_lens[:REQUESTS])
    layer.step(plan, x[:0], ids[:0], qkv[:0], q[:0], attended[:0], y[:0])   # library set-up stays out of the graph
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                 # and so does the products' first call at this size
        torch.matmul(x, layer.w_qkv.t(), out=qkv)
        torch.matmul(attended, layer.w_o.t(), out=y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    for _ in range(decode_steps):
        x.normal_()
        graph.replay()
        check(x, y, [1] * REQUESTS)
    # request 1 ends; its place goes to a new request in the step after, in pages that came back
    eager_step([1, -1, 1, 1])
    history[1], slots_of[1] = history[1][:0], 2
    eager_step([1, 33, 1, 2])
    # too few pages for request 3, also in the step in which request 0's come back; then there are
    eager_step([40, 30, 1, 40])
    eager_step([-1, 1, 1, 40])
    history[0] = history[0][:0]
    assert refusals == 2, "request 3 was to be refused twice"
    eager_step([16, 1, 1, 40])
    assert refusals == 2, "request 3 was to get its pages"
    held = sum(-(-len(h) // PAGE) for h in history)
    assert plan.query()["free_pages"] == PAGES - held, "pages lost"
    print(f"paged serving ok: lengths {[len(h) for h in history]}, {plan.query()['free_pages']} of {PAGES} pages free, "
          f"largest error {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
