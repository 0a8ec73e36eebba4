// Drives the paged-cache host code (kv.cpp) and the index arithmetic of its kernels
// (kv_index.h) under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU, together
// with hip_stubs.cpp: every refusal of the calls, and a host walk of the page plan's and
// the attention's addressing with wrong lengths and pages.  Test infrastructure only.
#include <climits>
#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

#include "kv.h"
#include "raxlora.h"

extern int g_launches;
namespace rax {
hipError_t launch_page_plan(const PagePlanArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
hipError_t launch_rotary_append(const RotaryArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
hipError_t launch_paged_attention(const AttentionArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
}  // namespace rax

extern "C" hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 8;
  return hipSuccess;
}

static int failures = 0;
#define EXPECT(call, want)                                                                                \
  do {                                                                                                    \
    const int got_ = (call);                                                                              \
    if (got_ != (want)) {                                                                                 \
      std::printf("line %d: %s = %d, want %d (%s)\n", __LINE__, #call, got_, (want), lora_last_error());   \
      ++failures;                                                                                         \
    }                                                                                                     \
  } while (0)
#define TRUE(c) EXPECT((c) ? 1 : 0, 1)

alignas(16) static int32_t ints[4096];
alignas(16) static char mem[1 << 16];

static lora_kv_cache cache() {
  lora_kv_cache c{};
  c.k = mem;
  c.v = mem;
  c.num_pages = 4;
  c.page_size = 16;
  c.num_heads = 2;
  c.head_dim = 32;
  c.head_stride = 32;
  c.token_stride = 64;
  c.page_stride = 1024;
  c.dtype = LORA_BF16;
  c.k_scale = c.v_scale = 1.f;
  return c;
}

static void plan_refusals() {
  auto call = [](int seqs, int tokens, int ps, int np, int ld, int mp) {
    return lora_page_plan(0, ints, ints, seqs, tokens, ps, np, ints, ints, ints, ints, ld, mp, ints, ints, ints, ints, ints,
                          nullptr);
  };
  const int n0 = g_launches;
  EXPECT(call(-1, 0, 16, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(LORA_MAX_SEQS + 1, 0, 16, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, -1, 16, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 8, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 24, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 2048, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 0, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, -16, 4, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 16, 0, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 16, 1 << 27, 4, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 16, 4, 3, 4), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 16, 4, 4, 0), LORA_ERR_SHAPE);
  EXPECT(call(1, 1, 16, 4, 1 << 28, 1 << 27), LORA_ERR_SHAPE);
  EXPECT(lora_page_plan(0, nullptr, ints, 1, 0, 16, 4, ints, ints, ints, ints, 4, 4, ints, ints, ints, ints, ints, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(lora_page_plan(0, ints, ints, 1, 1, 16, 4, ints, ints, ints, ints, 4, 4, ints, ints, nullptr, ints, ints, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(lora_page_plan(0, ints, ints, 1, 1, 16, 4, nullptr, ints, ints, ints, 4, 4, ints, ints, ints, ints, ints, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(lora_page_plan(0, ints, ints, 1, 1, 16, 4, ints, ints, ints, ints, 4, 4, ints, ints, ints, ints, nullptr, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(g_launches, n0);
  EXPECT(lora_page_plan(0, nullptr, nullptr, 0, 0, 16, 4, ints, ints, ints, nullptr, 4, 4, nullptr, ints, nullptr, nullptr, ints,
                        nullptr), LORA_OK);
  EXPECT(call(3, 5, 1024, 4, 4, 4), LORA_OK);
  EXPECT(g_launches, n0 + 2);
}

static void cache_refusals() {
  double f[16];
  for (double& x : f) x = 0.5;
  lora_rotary* r = nullptr;
  EXPECT(lora_rotary_create(nullptr, 0, 32, 0, f, 1.0), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_create(&r, 0, 32, 0, nullptr, 1.0), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_create(&r, 0, 31, 0, f, 1.0), LORA_ERR_SHAPE);
  EXPECT(lora_rotary_create(&r, 0, 0, 0, f, 1.0), LORA_ERR_SHAPE);
  EXPECT(lora_rotary_create(&r, 0, 258, 0, f, 1.0), LORA_ERR_SHAPE);
  EXPECT(lora_rotary_create(&r, 0, 32, 0, f, NAN), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_create(&r, 0, 32, 0, f, 1e300), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_create(&r, 5, 32, 0, f, 1.0), LORA_ERR_NO_DEVICE);
  f[3] = INFINITY;
  EXPECT(lora_rotary_create(&r, 0, 32, 0, f, 1.0), LORA_ERR_INVALID_ARG);
  f[3] = 0.5;
  TRUE(r == nullptr);
  EXPECT(lora_rotary_create(&r, 0, 32, 0, f, 1.0), LORA_OK);

  lora_attention* a = nullptr;
  EXPECT(lora_attention_create(nullptr, 0, 4, 8, 4, 2, 32), LORA_ERR_INVALID_ARG);
  EXPECT(lora_attention_create(&a, 0, 0, 8, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, LORA_MAX_SEQS + 1, 8, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, 4, 0, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, 4, 1 << 24, 1024, 1, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 5, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 4, 0, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 2048, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 4, 2, 40), LORA_ERR_ALIGN);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 4, 2, 0), LORA_ERR_ALIGN);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 4, 2, 272), LORA_ERR_SHAPE);
  EXPECT(lora_attention_create(&a, 3, 4, 8, 4, 2, 32), LORA_ERR_NO_DEVICE);
  TRUE(a == nullptr);
  EXPECT(lora_attention_create(&a, 0, 4, 8, 4, 2, 32), LORA_OK);

  auto append = [&](const lora_kv_cache& c, int ldx = 256, int hq = 4, lora_dtype dt = LORA_BF16, int T = 3, int ldq = 128,
                    void* x = mem) {
    return lora_rotary_append(r, x, ldx, dt, hq, ints, ints, T, mem, ldq, &c, nullptr);
  };
  auto attend = [&](const lora_kv_cache& c, int ldq = 128, lora_dtype dt = LORA_BF16, int ns = 2, int T = 3, float scale = 1.f,
                    int window = 0, int ld = 8, int mp = 8, void* q = mem) {
    return lora_paged_attention(a, q, ldq, dt, &c, ints, ld, mp, ints, ints, ns, T, scale, window, mem, 128, nullptr, nullptr);
  };
  const int n0 = g_launches;
  auto both = [&](const lora_kv_cache& c, int want) {
    EXPECT(append(c), want);
    EXPECT(attend(c), want);
  };
  lora_kv_cache c = cache();
  EXPECT(lora_rotary_append(nullptr, mem, 256, LORA_BF16, 4, ints, ints, 3, mem, 128, &c, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_append(r, mem, 256, LORA_BF16, 4, ints, ints, 3, mem, 128, nullptr, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_append(r, mem, 256, LORA_BF16, 4, nullptr, ints, 3, mem, 128, &c, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(lora_paged_attention(nullptr, mem, 128, LORA_BF16, &c, ints, 8, 8, ints, ints, 1, 1, 1.f, 0, mem, 128, nullptr, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(lora_paged_attention(a, mem, 128, LORA_BF16, &c, nullptr, 8, 8, ints, ints, 1, 1, 1.f, 0, mem, 128, nullptr, nullptr),
         LORA_ERR_INVALID_ARG);
  c.k = nullptr; both(c, LORA_ERR_INVALID_ARG); c = cache();
  c.k = mem + 8; both(c, LORA_ERR_ALIGN); c = cache();
  c.dtype = 9; both(c, LORA_ERR_DTYPE); c = cache();
  c.dtype = LORA_F32; both(c, LORA_ERR_DTYPE); c = cache();
  c.dtype = LORA_FP8E4M3; c.k_scale = 0.f; both(c, LORA_ERR_INVALID_ARG);
  c.k_scale = NAN; both(c, LORA_ERR_INVALID_ARG);
  c.k_scale = 1.f; c.v_scale = INFINITY; both(c, LORA_ERR_INVALID_ARG); c = cache();
  c.page_size = 12; both(c, LORA_ERR_SHAPE); c = cache();
  c.num_pages = 0; both(c, LORA_ERR_SHAPE); c = cache();
  c.num_pages = 1 << 28; both(c, LORA_ERR_SHAPE); c = cache();
  c.num_heads = 0; both(c, LORA_ERR_SHAPE); c = cache();
  c.head_dim = 24; both(c, LORA_ERR_ALIGN); c = cache();
  c.head_dim = 512; both(c, LORA_ERR_SHAPE); c = cache();
  c.head_stride = 16; both(c, LORA_ERR_SHAPE); c = cache();       // heads overlap
  c.token_stride = 32; both(c, LORA_ERR_SHAPE); c = cache();      // tokens on the heads
  c.token_stride = -64; both(c, LORA_ERR_SHAPE); c = cache();
  c.page_stride = 512; both(c, LORA_ERR_SHAPE); c = cache();
  c.page_stride = LLONG_MAX - 15; both(c, LORA_ERR_SHAPE); c = cache();
  c.page_stride = 1032; both(c, LORA_ERR_ALIGN); c = cache();
  c.token_stride = 1 << 25; c.page_stride = 1LL << 30; both(c, LORA_ERR_SHAPE); c = cache();
  EXPECT(append(c, 248), LORA_ERR_SHAPE);
  EXPECT(append(c, 260), LORA_ERR_ALIGN);
  EXPECT(append(c, 256, 3), LORA_ERR_SHAPE);
  EXPECT(append(c, 256, 0), LORA_ERR_SHAPE);
  EXPECT(append(c, 256, 4, LORA_FP8E4M3), LORA_ERR_DTYPE);
  EXPECT(append(c, 256, 4, LORA_F32), LORA_ERR_DTYPE);
  EXPECT(append(c, 256, 4, LORA_BF16, -1), LORA_ERR_SHAPE);
  EXPECT(append(c, 256, 4, LORA_BF16, 3, 120), LORA_ERR_SHAPE);
  EXPECT(append(c, 256, 4, LORA_BF16, 3, 128, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(append(c, 256, 4, LORA_BF16, 3, 128, mem + 4), LORA_ERR_ALIGN);
  EXPECT(attend(c, 120), LORA_ERR_SHAPE);
  EXPECT(attend(c, 132), LORA_ERR_ALIGN);
  EXPECT(attend(c, 128, LORA_F32), LORA_ERR_DTYPE);
  EXPECT(attend(c, 128, LORA_BF16, 5), LORA_ERR_CAPACITY);
  EXPECT(attend(c, 128, LORA_BF16, 2, 9), LORA_ERR_CAPACITY);
  EXPECT(attend(c, 128, LORA_BF16, -1), LORA_ERR_SHAPE);
  EXPECT(attend(c, 128, LORA_BF16, 2, 3, NAN), LORA_ERR_INVALID_ARG);
  EXPECT(attend(c, 128, LORA_BF16, 2, 3, 1.f, -1), LORA_ERR_INVALID_ARG);
  EXPECT(attend(c, 128, LORA_BF16, 2, 3, 1.f, 0, 7), LORA_ERR_SHAPE);
  EXPECT(attend(c, 128, LORA_BF16, 2, 3, 1.f, 0, 8, 0), LORA_ERR_SHAPE);
  EXPECT(attend(c, 128, LORA_BF16, 2, 3, 1.f, 0, 8, 8, nullptr), LORA_ERR_INVALID_ARG);
  c.num_heads = 1; EXPECT(attend(c), LORA_ERR_SHAPE); c = cache();
  c.head_dim = 16; c.head_stride = 16; EXPECT(append(c), LORA_ERR_SHAPE);   // rot_dim above the head
  c = cache();
  EXPECT(g_launches, n0);
  EXPECT(append(c), LORA_OK);
  EXPECT(attend(c), LORA_OK);
  c.dtype = LORA_FP8E4M3;
  EXPECT(append(c), LORA_OK);
  EXPECT(attend(c), LORA_OK);
  c = cache();
  c.token_stride = 32; c.head_stride = 512;                                 // heads outside the tokens
  EXPECT(append(c), LORA_OK);
  EXPECT(attend(c), LORA_OK);
  c = cache();
  c.num_pages = 1; c.num_heads = 2; c.page_stride = 0;                      // the stride of a single page is free
  EXPECT(append(c), LORA_OK);
  EXPECT(g_launches, n0 + 7);
  EXPECT(append(c, 256, 4, LORA_BF16, 0), LORA_OK);
  EXPECT(attend(cache(), 128, LORA_BF16, 2, 0), LORA_OK);
  EXPECT(g_launches, n0 + 7);                                               // nothing to do: nothing launched
  EXPECT(lora_rotary_destroy(r), LORA_OK);
  EXPECT(lora_rotary_destroy(nullptr), LORA_OK);
  EXPECT(lora_attention_destroy(a), LORA_OK);
  EXPECT(lora_attention_destroy(nullptr), LORA_OK);
}

static void frequency_refusals() {
  double f[LORA_MAX_HEAD_DIM / 2];
  EXPECT(lora_rotary_frequencies(64, 1e4, LORA_ROPE_PLAIN, 0, 0, 0, 0, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_frequencies(63, 1e4, LORA_ROPE_PLAIN, 0, 0, 0, 0, f), LORA_ERR_SHAPE);
  EXPECT(lora_rotary_frequencies(64, 1.0, LORA_ROPE_PLAIN, 0, 0, 0, 0, f), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_frequencies(64, NAN, LORA_ROPE_PLAIN, 0, 0, 0, 0, f), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_frequencies(64, 1e4, 4, 1, 0, 0, 0, f), LORA_ERR_SHAPE);
  EXPECT(lora_rotary_frequencies(64, 1e4, LORA_ROPE_LINEAR, 0.5, 0, 0, 0, f), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_frequencies(64, 1e4, LORA_ROPE_WAVELENGTH, 8, 0, 1, 4, f), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_frequencies(64, 1e4, LORA_ROPE_DIM, 8, 4096, 32, 1, f), LORA_ERR_INVALID_ARG);
  EXPECT(lora_rotary_frequencies(256, 1e4, LORA_ROPE_DIM, 8, 4096, 1, 32, f), LORA_OK);
  EXPECT(lora_rotary_frequencies(2, 1e4, LORA_ROPE_DIM, 8, 1e-3, 1, 32, f), LORA_OK);
}

// every index the kernels form from a request's or a sequence's words stays in its range
static void index_walk() {
  std::mt19937 g(7);
  const int odd[] = {INT_MIN, -1000, -2, -1, 0, 1, 15, 16, 17, 100, 1 << 20, 1 << 30, INT_MAX - 1, INT_MAX};
  const int n_odd = sizeof odd / sizeof *odd;
  for (int shift : {4, 6, 10})
    for (int max_pages : {1, 7, INT_MAX >> 10})
      for (int past : odd)
        for (int fresh : odd) {
          if (((long long)max_pages << shift) > INT_MAX) continue;
          const rax::RequestNeed q = rax::request_need(past, fresh, shift, max_pages);
          TRUE(q.n >= 0 && q.n <= rax::kPlanCap && q.have >= 0 && q.need >= 0 && q.back >= 0);
          TRUE((long long)q.have + q.need <= max_pages && q.back <= max_pages);
          TRUE(!(q.live && q.invalid) && (q.back == 0 || !q.live));
          if (q.live && q.n > 0) TRUE(((past + q.n - 1) >> shift) < q.have + q.need);
          if (q.live) TRUE(past + q.n >= 0);
        }
  for (int n : {1, 2, 1000, INT_MAX})
    for (int h : odd) {
      const int head = rax::ring_head(h, n);
      TRUE(head >= 0 && head < n);
      for (int off : {0, 1, n / 2, n - 1}) TRUE(rax::ring_at(head, off, n) >= 0 && rax::ring_at(head, off, n) < n);
    }
  for (int a : odd)
    for (int b : odd)
      if (a >= 0 && b >= 0 && a <= rax::kPlanCap && b <= rax::kPlanCap) {
        const long long want = std::min<long long>((long long)a + b, rax::kPlanCap);
        TRUE(rax::sat_add(a, b) == want);
      }
  for (int page : odd) {
    const int p = rax::page_or_none(page, 17);
    TRUE(p == -1 || (p >= 0 && p < 17 && p == page));
  }
  for (int i = 0; i < 20000; ++i) {
    const int T = 1 + g() % 50, max_len = 16 * (1 + g() % 8);
    auto word = [&]() { return g() % 2 ? odd[g() % n_odd] : (int)(g() % 60) - 5; };
    const rax::SeqRows s = rax::seq_rows(word(), word(), word(), T, max_len);
    TRUE(s.start >= 0 && s.n >= 0 && s.start + s.n <= T && s.len >= 0 && s.len <= max_len);
    const int window = g() % 3 ? (int)(g() % 40) : odd[g() % n_odd] < 0 ? 0 : odd[g() % n_odd];
    for (int t = 0; t < s.n; ++t) {
      const rax::KeyRange k = rax::token_keys(t, s.n, s.len, window < 0 ? 0 : window);
      TRUE(k.lo >= 0 && k.hi >= 0 && k.hi <= s.len);
      for (int j = 0; j < max_len; ++j) {   // the definition
        const int pos = s.len - s.n + t;
        const bool see = j <= pos && (window <= 0 || j > (long long)pos - window);
        TRUE(see == (j >= k.lo && j < k.hi));
      }
    }
  }
}

// the attention's line of steps: equal contiguous shares that cover it once, and the spans
// of the sequences that make it up
static void share_walk() {
  std::mt19937 g(11);
  for (int i = 0; i < 3000; ++i) {
    const int work = 1 + (int)(i % 3 ? g() % 500 : g() % INT_MAX);
    const int n = 1 + (int)(g() % std::min(work, 512));
    TRUE(rax::share_start(work, n, 0) == 0 && rax::share_start(work, n, n) == work);
    for (int b = 0; b < n; ++b) {
      const int x0 = rax::share_start(work, n, b), x1 = rax::share_start(work, n, b + 1);
      TRUE(x1 > x0 && x1 - x0 <= work / n + 1);
      TRUE(rax::share_owner(work, n, x0) == b && rax::share_owner(work, n, x1 - 1) == b);
    }
  }
  for (int i = 0; i < 20000; ++i) {
    const int max_len = i % 2 ? 16 * (1 + (int)(g() % 40)) : INT_MAX / 16 * 16, T = 1 + (int)(g() % 50);
    const rax::SeqRows s = rax::seq_rows((int)(g() % 60), (int)(g() % 60), (int)(g() % 3 ? g() % 700 : g()), T, max_len);
    const int window = g() % 2 ? 0 : (int)(g() % 3 ? g() % 300 : g() >> 1), step_log2 = 4 + g() % 5, step = 1 << step_log2;
    const rax::SeqSpan x = rax::seq_span(s, window, step_log2);
    TRUE((x.steps == 0) == (s.n == 0) && x.base % 16 == 0);
    for (int t = 0; t < s.n; ++t) {
      const rax::KeyRange k = rax::token_keys(t, s.n, s.len, window);
      if (k.hi > k.lo) TRUE((unsigned)k.lo >= x.base && (unsigned)k.hi <= x.base + (unsigned long long)x.steps * step);
    }
    if (x.steps > 1) TRUE(x.base + (unsigned long long)(x.steps - 1) * step < (unsigned)s.len);
  }
  for (int d = 1; d <= 1024; ++d) {
    const rax::FastDiv f = rax::fast_div(d);
    for (int n : {0, 1, d - 1, d, d + 1, 5 * d - 1, 5 * d, 12345 * d - 1, 12345 * d, (1 << 30) / d * d, (1 << 30) / d * d - 1,
                  1 << 30, INT_MAX, INT_MAX / d * d - 1, INT_MAX / d * d})
      TRUE(rax::fast_quot(n, f) == n / d);
  }
  for (int i = 0; i < 3000; ++i) {   // the line stays below the cap, also with every key and token there is
    const int seqs = 1 + g() % LORA_MAX_SEQS, group = 1 + g() % 64, heads = 1 + g() % (1024 / group), rows_log2 = 4 + g() % 3;
    const int T = 1 + (int)(g() % (g() % 2 ? 70000 : 1 << 24)), max_len = 1 + (int)(g() % (g() % 2 ? 1 << 20 : INT_MAX));
    const int step = rax::line_step_log2(5, seqs, T, max_len, heads, group, rows_log2);
    TRUE(step == -1 || (step >= 5 && step <= 30));
    if (step < 0) {   // refused: there are that many units
      TRUE(((double)rax::row_blocks(T, group, rows_log2) + seqs) * heads * 4.0 >= rax::kPlanCap);
      continue;
    }
    double line = 0;
    for (int r = 0; r < seqs; ++r) {   // tokens dealt evenly, all sequences of the longest length
      const int n = T / seqs + (r < T % seqs);
      const rax::SeqSpan x = rax::seq_span(rax::SeqRows{0, n, max_len}, 0, step);
      line += (double)x.steps * heads * rax::row_blocks(n, group, rows_log2);
    }
    TRUE(line < rax::kPlanCap);
  }
  for (long long rows : {1LL, 16LL, 17LL, 33LL, 65LL, 1LL << 30})
    for (long long heads : {1LL, 64LL, 128LL, 4096LL * 1024}) {
      const rax::AttnRows r = rax::attention_rows(rows, heads);
      TRUE(4 % r.waves == 0 && r.rows() <= rax::kMaxRows && (r.rows() == 16 || 2 * rows > r.rows()));
    }
}

int main() {
  share_walk();
  plan_refusals();
  cache_refusals();
  frequency_refusals();
  index_walk();
  std::printf("%d failures\n", failures);
  return failures != 0;
}
