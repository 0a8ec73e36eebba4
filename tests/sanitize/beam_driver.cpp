// Drives the host code of the beam search operators (beam.cpp, shared.cpp) and the index arithmetic of their kernels
// (fork_index.h, shared_index.h) under AddressSanitizer and UndefinedBehaviorSanitizer on the CPU, together with
// hip_stubs.cpp: every refusal of the calls, and host walks of the fork's columns and of the shared attention's two
// lines, their shares and the parts that the merge joins.  Test infrastructure only.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <map>
#include <random>
#include <vector>

#include "beam.h"
#include "fork_index.h"
#include "raxlora.h"
#include "shared.h"

extern int g_launches;
static rax::SharedArgs g_shared;
static rax::BeamArgs g_beam;
static int g_cus = 256;
namespace rax {
hipError_t launch_beam_select(const BeamArgs& a, hipStream_t, const KTimer&) { ++g_launches; g_beam = a; return hipSuccess; }
hipError_t launch_page_fork(const PageForkArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
hipError_t launch_page_copy(const PageCopyArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
hipError_t launch_shared_attention(const SharedArgs& s, hipStream_t, const KTimer&) { ++g_launches; g_shared = s; return hipSuccess; }
hipError_t launch_shared_merge(const SharedArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
}  // namespace rax

extern "C" hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = g_cus;
  return hipSuccess;
}

static int failures = 0;
#define EXPECT(call, want)                                                                                \
  do {                                                                                                    \
    const int got_ = (call);                                                                              \
    if (got_ != (want)) {                                                                                 \
      if (failures < 40) std::printf("line %d: %s = %d, want %d (%s)\n", __LINE__, #call, got_, (want), lora_last_error()); \
      ++failures;                                                                                         \
    }                                                                                                     \
  } while (0)
#define TRUE(c) EXPECT((c) ? 1 : 0, 1)

alignas(16) static int32_t v[12][4096];   // vectors that do not overlap
alignas(16) static float fl[4][4096];
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

static void select_refusals() {
  lora_beams* b = nullptr;
  EXPECT(lora_beams_create(nullptr, 0, 4, 4, 100, 4), LORA_ERR_INVALID_ARG);
  for (int bad : {0, -1, LORA_MAX_SEQS + 1}) EXPECT(lora_beams_create(&b, 0, bad, 4, 100, 4), LORA_ERR_SHAPE);
  for (int bad : {0, -1, LORA_MAX_BEAMS + 1}) {
    EXPECT(lora_beams_create(&b, 0, 4, bad, 100, 4), LORA_ERR_SHAPE);
    EXPECT(lora_beams_create(&b, 0, 4, 4, 100, bad), LORA_ERR_SHAPE);
  }
  for (int bad : {0, -1, LORA_MAX_VOCAB + 1}) EXPECT(lora_beams_create(&b, 0, 4, 4, bad, 4), LORA_ERR_SHAPE);
  EXPECT(lora_beams_create(&b, 7, 4, 4, 100, 4), LORA_ERR_NO_DEVICE);
  TRUE(b == nullptr);
  EXPECT(lora_beams_create(&b, 0, 4, 4, 100, 4), LORA_OK);
  const int n0 = g_launches;
  auto call = [&](const void* x = mem, int ld = 100, lora_dtype dt = LORA_BF16, const int32_t* ended = v[0], int end = 5, int n = 2,
                  int32_t* parents = v[1], int32_t* tokens = v[2], float* out = fl[1], int32_t* ended_out = v[3], const float* wt = fl[2],
                  const float* scores = fl[0]) {
    return lora_beam_select(b, x, ld, dt, scores, ended, end, wt, n, parents, tokens, out, ended_out, nullptr);
  };
  EXPECT(lora_beam_select(nullptr, mem, 100, LORA_BF16, fl[0], nullptr, -1, nullptr, 1, v[1], v[2], fl[1], nullptr, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 99), LORA_ERR_SHAPE);
  EXPECT(call(mem, 100, LORA_FP8E4M3), LORA_ERR_DTYPE);
  EXPECT(call(mem + 1), LORA_ERR_ALIGN);
  EXPECT(call(mem + 2, 100, LORA_F32), LORA_ERR_ALIGN);
  EXPECT(call(mem, 100, LORA_BF16, v[0], -1), LORA_ERR_INVALID_ARG);      // ended rows need a token
  EXPECT(call(mem, 100, LORA_BF16, nullptr, -2), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 100), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, -1), LORA_ERR_SHAPE);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 5), LORA_ERR_CAPACITY);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[2], nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[1]), LORA_ERR_INVALID_ARG);           // two outputs
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[1] + 7), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[0]), LORA_ERR_INVALID_ARG);                 // parents on ended
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[2], fl[2]), LORA_ERR_INVALID_ARG);    // scores_out on weights
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[2], fl[0] + 1), LORA_ERR_INVALID_ARG);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[2], fl[1], v[0] + 1), LORA_ERR_INVALID_ARG);
  EXPECT(g_launches, n0);
  EXPECT(call(), LORA_OK);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[2], fl[0], v[0]), LORA_OK);           // in place
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[1] + 8), LORA_OK);                    // side by side
  EXPECT(call(mem, 100, LORA_F32, nullptr, -1, 4, v[1], v[2], fl[1], nullptr, nullptr), LORA_OK);
  EXPECT(g_launches, n0 + 4);
  EXPECT(call(nullptr, 100, LORA_BF16, nullptr, -1, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), LORA_OK);
  EXPECT(g_launches, n0 + 4);
  EXPECT(lora_beams_destroy(b), LORA_OK);
  EXPECT(lora_beams_destroy(nullptr), LORA_OK);
  EXPECT(lora_beams_create(&b, 0, 4, 4, 100, 3), LORA_OK);                                   // fewer candidates than beams
  EXPECT(call(), LORA_OK);
  EXPECT(call(mem, 100, LORA_BF16, v[0], 5, 2, v[1], v[2], fl[0]), LORA_ERR_INVALID_ARG);    // not in place then
  EXPECT(lora_beams_destroy(b), LORA_OK);
}

static void fork_refusals() {
  const int n0 = g_launches;
  auto call = [](int rows, int ps = 16, int np = 40, int ld = 4, int mp = 4, int a = -1, int b = 0) {
    int32_t* p[11];
    for (int i = 0; i < 11; ++i) p[i] = v[i];
    if (a >= 0) p[a] = b < 0 ? nullptr : p[b] + 1;
    return lora_page_fork(0, p[0], rows, p[1], ps, np, p[2], p[3], p[4], p[5], ld, mp, p[6], p[7], p[8], p[9], p[10], nullptr);
  };
  EXPECT(call(-1), LORA_ERR_SHAPE);
  EXPECT(call(LORA_MAX_SEQS + 1), LORA_ERR_SHAPE);
  for (int bad : {0, -16, 8, 24, 2048}) EXPECT(call(3, bad), LORA_ERR_SHAPE);
  EXPECT(call(3, 16, 0), LORA_ERR_SHAPE);
  EXPECT(call(3, 16, 1 << 27), LORA_ERR_SHAPE);
  EXPECT(call(3, 16, 40, 3), LORA_ERR_SHAPE);
  EXPECT(call(3, 16, 40, 4, 0), LORA_ERR_SHAPE);
  EXPECT(call(3, 16, 40, 1 << 28, 1 << 27), LORA_ERR_SHAPE);
  for (int i = 0; i < 11; ++i) EXPECT(call(3, 16, 40, 4, 4, i, -1), LORA_ERR_INVALID_ARG);
  for (int i = 0; i < 11; ++i)      // any vector that begins inside another
    for (int j = 0; j < 11; ++j)
      if (i != j) EXPECT(call(40, 16, 400, 4, 4, i, j), LORA_ERR_INVALID_ARG);
  EXPECT(g_launches, n0);
  EXPECT(call(3), LORA_OK);
  EXPECT(call(0), LORA_OK);
  EXPECT(lora_page_fork(0, nullptr, 0, nullptr, 16, 40, v[2], v[3], v[4], nullptr, 4, 4, nullptr, nullptr, nullptr, v[9], v[10], nullptr), LORA_OK);
  EXPECT(g_launches, n0 + 1);
}

static void copy_refusals() {
  const int n0 = g_launches;
  std::vector<lora_kv_cache> l(LORA_MAX_LAYERS + 1, cache());
  auto call = [&](int layers, int pairs = 3, const int32_t* src = v[0], const int32_t* dst = v[1]) {
    return lora_page_copy(0, l.data(), layers, src, dst, v[2], pairs, nullptr);
  };
  EXPECT(lora_page_copy(0, nullptr, 1, v[0], v[1], nullptr, 1, nullptr), LORA_ERR_INVALID_ARG);
  for (int bad : {0, -1, LORA_MAX_LAYERS + 1}) EXPECT(call(bad), LORA_ERR_SHAPE);
  for (int bad : {-1, (1 << 20) + 1}) EXPECT(call(2, bad), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(2, 3, v[0], nullptr), LORA_ERR_INVALID_ARG);
  l[1].page_size = 32; l[1].page_stride = 2048; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].page_stride = 2048; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].token_stride = 128; l[1].page_stride = 2048; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].num_pages = 3; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].head_dim = 16; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].num_heads = 1; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].dtype = LORA_FP8E4M3; EXPECT(call(2), LORA_ERR_SHAPE); l[1] = cache();
  l[1].k = nullptr; EXPECT(call(2), LORA_ERR_INVALID_ARG); l[1] = cache();
  l[1].v = mem + 4; EXPECT(call(2), LORA_ERR_ALIGN); l[1] = cache();
  l[0].page_stride = 512; EXPECT(call(1), LORA_ERR_SHAPE); l[0] = cache();
  EXPECT(g_launches, n0);
  l[1].k = mem + 4096;
  EXPECT(call(2), LORA_OK);
  EXPECT(call(LORA_MAX_LAYERS), LORA_OK);
  EXPECT(call(1, 0, nullptr, nullptr), LORA_OK);
  EXPECT(g_launches, n0 + 2);
}

static void shared_refusals() {
  lora_shared* a = nullptr;
  EXPECT(lora_shared_create(nullptr, 0, 4, 8, 4, 2, 32), LORA_ERR_INVALID_ARG);
  EXPECT(lora_shared_create(&a, 0, 0, 8, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, LORA_MAX_SEQS + 1, 8, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, 4, 0, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, 4, (1 << 24) + 1, 4, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, 4, 1 << 24, 1024, 1, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, 4, 8, 5, 2, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, 4, 8, 4, 0, 32), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 0, 4, 8, 4, 2, 40), LORA_ERR_ALIGN);
  EXPECT(lora_shared_create(&a, 0, 4, 8, 4, 2, 272), LORA_ERR_SHAPE);
  EXPECT(lora_shared_create(&a, 3, 4, 8, 4, 2, 32), LORA_ERR_NO_DEVICE);
  TRUE(a == nullptr);
  EXPECT(lora_shared_create(&a, 0, 4, 8, 4, 2, 32), LORA_OK);
  const int n0 = g_launches;
  lora_kv_cache c = cache();
  auto call = [&](int ns = 2, int T = 3, int ng = 1, float scale = 1.f, int ld = 8, int mp = 8, const int32_t* gs = v[3],
                  const int32_t* cm = v[4], lora_dtype dt = LORA_BF16, int ldq = 128, void* q = mem, int ldo = 128, const int32_t* table = v[0]) {
    return lora_shared_attention(a, q, ldq, dt, &c, table, ld, mp, v[1], v[2], ns, T, gs, cm, ng, scale, mem + 8192, ldo, nullptr, nullptr);
  };
  EXPECT(lora_shared_attention(nullptr, mem, 128, LORA_BF16, &c, v[0], 8, 8, v[1], v[2], 1, 1, v[3], v[4], 1, 1.f, mem, 128, nullptr, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(lora_shared_attention(a, mem, 128, LORA_BF16, nullptr, v[0], 8, 8, v[1], v[2], 1, 1, v[3], v[4], 1, 1.f, mem, 128, nullptr, nullptr),
         LORA_ERR_INVALID_ARG);
  EXPECT(call(-1), LORA_ERR_SHAPE);
  EXPECT(call(5), LORA_ERR_CAPACITY);
  EXPECT(call(2, -1), LORA_ERR_SHAPE);
  EXPECT(call(2, 9), LORA_ERR_CAPACITY);
  EXPECT(call(2, 3, -1), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, 5), LORA_ERR_CAPACITY);
  EXPECT(call(2, 3, 1, NAN), LORA_ERR_INVALID_ARG);
  EXPECT(call(2, 3, 1, INFINITY), LORA_ERR_INVALID_ARG);
  EXPECT(call(2, 3, 1, 1.f, 7), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, 1, 1.f, 8, 0), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, 1, 1.f, 1 << 28, 1 << 27), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_F32), LORA_ERR_DTYPE);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_BF16, 120), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_BF16, 132), LORA_ERR_ALIGN);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_BF16, 128, nullptr), LORA_ERR_INVALID_ARG);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_BF16, 128, mem + 4), LORA_ERR_ALIGN);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_BF16, 128, mem, 120), LORA_ERR_SHAPE);
  EXPECT(call(2, 3, 1, 1.f, 8, 8, v[3], v[4], LORA_BF16, 128, mem, 128, nullptr), LORA_ERR_INVALID_ARG);
  c.head_dim = 16; EXPECT(call(), LORA_ERR_SHAPE); c = cache();
  c.num_heads = 1; EXPECT(call(), LORA_ERR_SHAPE); c = cache();
  c.page_stride = 512; EXPECT(call(), LORA_ERR_SHAPE); c = cache();
  EXPECT(g_launches, n0);
  EXPECT(call(), LORA_OK);
  EXPECT(call(2, 3, 0, 1.f, 8, 8, nullptr, nullptr), LORA_OK);
  EXPECT(g_launches, n0 + 4);
  EXPECT(call(0), LORA_OK);
  EXPECT(call(2, 0), LORA_OK);
  EXPECT(g_launches, n0 + 4);
  EXPECT(lora_shared_destroy(a), LORA_OK);
  EXPECT(lora_shared_destroy(nullptr), LORA_OK);
}

// the shapes of a call for all sizes: tables and tiles fit into LDS, the lines stay below the cap
static void shape_walk() {
  std::mt19937 g(5);
  for (int i = 0; i < 400; ++i) {
    const int group = 1 + (int)(g() % 3 ? g() % 8 : g() % 64), kv = 1 + g() % 8, dims[] = {16, 64, 96, 128, 192, 256}, dim = dims[g() % 6];
    const int ns = 1 + (int)(g() % 2 ? g() % 30 : g() % LORA_MAX_SEQS), T = (int)(ns + g() % 2000), ng = (int)(g() % 3 ? g() % (ns + 1) : 1);
    lora_shared* a = nullptr;
    EXPECT(lora_shared_create(&a, 0, ns, T, group * kv, kv, dim), LORA_OK);
    lora_kv_cache c = cache();
    const int type = g() % 3;
    c.dtype = type == 0 ? LORA_BF16 : type == 1 ? LORA_FP8E4M3 : LORA_F32;
    c.num_heads = kv;
    c.head_dim = c.head_stride = dim;
    c.token_stride = kv * dim;
    c.page_stride = 16 * kv * dim;
    const int width = group * kv * dim;
    const int mp = g() % 2 ? 1 << 10 : INT_MAX / 16;
    const int st = lora_shared_attention(a, mem, width, type == 2 ? LORA_F32 : LORA_BF16, &c, v[0], mp, mp, v[1], v[2], ns, T, v[3], v[4],
                                         ng, 1.f, mem, width, nullptr, nullptr);
    EXPECT(st, LORA_OK);
    const rax::SharedArgs& s = g_shared;
    const bool wide = s.common_line.row_waves == 4;
    if (wide) TRUE(s.common_line.rows_log2 == rax::kWideRowsLog2 && ng <= rax::kWideGroups && type != 2 && (dim == 64 || dim == 128));
    for (const rax::LineShape* l : {&s.common_line, &s.own_line}) {
      TRUE(1 << l->rows_log2 == (l == &s.common_line && wide ? 128 : 16 * l->row_tiles * std::max(1, l->row_waves)));
      if (dim > 128) TRUE(l->row_tiles == 1 && (l->row_waves == 2 || (l == &s.own_line && l->row_waves == 0)));
    }
    TRUE(s.own_line.min_steps >= 1 && s.common_line.min_steps >= 1 && s.a.workers % (2 * rax::kDies) == 0);
    // two tiles of keys and values, or the join's rows: at most 4 waves' 16 rows of 128 + 4 numbers and their statistics
    const long long lds = wide ? 4LL * 64 * dim * 2 : 4 * 16 * (128 + 4 + 4) * 4;
    TRUE(lds + 4LL * (2 * ns + 4 * ng + 1) + 512 <= 160 * 1024);
    // every share's two places lie in the workspace
    TRUE((long long)s.a.workers * (s.own_line.row_waves == 0 ? 4 : 1) << s.own_line.rows_log2 <= (long long)s.a.workers * rax::kMaxRows);
    EXPECT(lora_shared_destroy(a), LORA_OK);
  }
  for (int cus : {1, 7, 64, 256, 304}) {
    const int w = rax::attention_workers(cus);
    TRUE(w % (2 * rax::kDies) == 0 && w >= 2 * rax::kDies && w <= 512);
  }
  for (int i = 0; i < 20000; ++i) {   // beam selection: workgroups of a row
    const long long rows = 1 + (long long)(g() % 2 ? g() % 64 : g() % (LORA_MAX_SEQS * LORA_MAX_BEAMS));
    const int vocab = 1 + (int)(g() % 2 ? g() % 300000 : g() % LORA_MAX_VOCAB), size = g() % 2 ? 2 : 4;
    const int segs = rax::beam_segs(rows, vocab, size);
    const long long tiles = ((long long)vocab * size + 15 + rax::kBeamTileBytes - 1) / rax::kBeamTileBytes;
    TRUE(segs >= 1 && (segs - 1) * (long long)rax::kBeamWaves < tiles);
    TRUE((long long)std::min<long long>(rows, LORA_MAX_BEAMS) * segs <= rax::kBeamMaxLists);   // of a request
    if (segs > 1) TRUE(rows * segs * rax::kBeamWaves <= 3LL * rax::kBeamMaxWaves + rows * rax::kBeamWaves);
  }
}

static void fork_walk() {
  const int odd[] = {INT_MIN, -17, -1, 0, 1, 15, 16, 17, 31, 32, 1000, 1 << 20, INT_MAX - 1, INT_MAX};
  for (int shift : {4, 6, 10})
    for (int max_pages : {1, 2, 7, INT_MAX >> 10})
      for (int len : odd) {
        const rax::RowPages p = rax::row_pages(len, shift, max_pages);
        const bool in = len >= 0 && (long long)len <= (long long)max_pages << shift;
        TRUE(p.invalid == !in && p.full >= 0 && p.part >= 0 && p.part < 1 << shift && p.all() <= max_pages);
        if (in) TRUE(((long long)p.full << shift) + p.part == len);
        for (int c : {0, p.full - 1, p.full, p.full + 1})
          for (int kids : {0, 1, 2, 5}) {
            const int d = rax::holders_change(p, c, kids);
            // of the definition: holders after minus holders before, of the page at column c
            const int want = c < 0 ? d : c < p.full ? kids - 1 : c == p.full && p.part ? (kids ? 0 : -1) : 0;
            TRUE(c < 0 || d == want);
          }
      }
  for (int rows : {0, 1, 5, LORA_MAX_SEQS})
    for (int x : odd) {
      const int p = rax::parent_or_none(x, rows);
      TRUE(p == -1 || (p == x && p >= 0 && p < rows));
    }
  for (int strips = 1; strips <= 70; ++strips) {   // every strip has one workgroup
    std::vector<int> seen(strips, 0);
    for (int b = 0; b < rax::whole_dies(strips); ++b) {
      const int s = rax::strip_of_block(b, strips);
      TRUE(s >= 0 && s <= strips);
      if (s < strips) ++seen[s];
    }
    for (int x : seen) TRUE(x == 1);
  }
}

static void group_walk() {
  std::mt19937 g(3);
  const int odd[] = {INT_MIN, -5, -1, 0, 1, 16, 17, 100, 1 << 20, INT_MAX - 1, INT_MAX};
  for (int i = 0; i < 5000; ++i) {
    const int n = 1 + g() % 40, groups = g() % 9;
    std::vector<int> start(groups + 1);
    for (int& x : start) x = (int)(g() % (n + 1));
    const bool rising = i % 2;
    if (rising) std::sort(start.begin(), start.end());
    for (int r = 0; r < n; ++r) {
      const int x = rax::group_of(start.data(), groups, r);
      TRUE(x >= -1 && x < groups);
      if (x >= 0) TRUE(start[x] <= r && r < start[x + 1]);
      if (rising) {
        int want = -1;
        for (int k = 0; k < groups; ++k)
          if (start[k] <= r && r < start[k + 1]) want = k;
        TRUE(x == want);
      }
    }
  }
  for (int i = 0; i < 20000; ++i) {
    const int T = 1 + g() % 50, max_len = i % 5 ? 16 * (1 + (int)(g() % 20)) : INT_MAX / 16 * 16;
    auto word = [&]() { return g() % 4 == 0 ? odd[g() % 11] : (int)(g() % 300) - 5; };
    const rax::SeqRows s = rax::seq_rows(word(), word(), word(), T, max_len);
    const int common = word(), from = rax::own_from(s, common, max_len), step_log2 = 4 + g() % 5;
    TRUE(from >= 0 && from <= s.len && (from == 0 || (s.n > 0 && from <= s.len - s.n && from == std::min(common, max_len))));
    const rax::SeqSpan x = rax::own_span(s, from, step_log2);
    TRUE((x.steps == 0) == (s.n <= 0) && x.base % 16 == 0 && (int)x.base <= from);
    for (int t = 0; t < s.n; ++t) {
      const rax::KeyRange k = rax::own_keys(t, s, from), all = rax::token_keys(t, s.n, s.len, 0);
      TRUE(k.lo == from && k.hi == all.hi && (from == 0 || k.hi > k.lo));
      if (k.hi > k.lo) TRUE((unsigned)k.hi <= x.base + ((unsigned long long)x.steps << step_log2));
    }
    const rax::SeqSpan y = rax::common_span(s, step_log2);
    TRUE(y.base == 0 && (s.n <= 0 || s.len <= 0 ? y.steps == 0 : (unsigned long long)y.steps << step_log2 >= (unsigned)s.len));
    if (y.steps > 0) TRUE((unsigned long long)(y.steps - 1) << step_log2 < (unsigned)s.len);
  }
  for (int i = 0; i < 20000; ++i) {
    const int steps = (int)(g() % 3 ? g() % 600 : g() % (1 << 25)), most = 1 + (int)(g() % 2 ? g() % 80 : g() % (1 << 25));
    const rax::EvenParts p = rax::even_parts(steps, most);
    TRUE(steps == 0 ? p.parts == 0 : p.parts >= 1 && p.steps >= 1 && p.steps <= most && (long long)p.parts * p.steps >= steps &&
                                         (long long)(p.parts - 1) * p.steps < steps);
    const int workers = 1 + g() % 512, work = 1 + (int)(g() % (g() % 2 ? 40000 : rax::kPlanCap));
    int last = (work + workers - 1LL) / workers;
    TRUE(rax::even_most(work, workers, 0) == last);
    for (int k = 1; k < 64; ++k) {
      const int m = rax::even_most(work, workers, k);
      TRUE(m >= last && m <= rax::even_most(work, workers, 0) * 9LL / 8);
      last = m;
    }
  }
}

// Both lines' workgroups: each share of each line has one.
static void split_walk() {
  std::mt19937 g(4);
  for (int i = 0; i < 3000; ++i) {
    const int grid = 2 * rax::kDies * (1 + (int)(g() % 32)), cm = 1 + g() % 9, om = 1 + g() % 9;
    const int cw = g() % 4 ? (int)(g() % 6000) : 0, ow = 1 + g() % 6000;
    const rax::LineSplit s = rax::split_lines(cw, cm, ow, om, grid);
    TRUE(s.common >= (cw > 0) && s.own >= 1 && s.common <= grid && s.own <= grid && s.common <= cw && s.own <= ow);
    std::vector<int> c(s.common, 0), o(s.own, 0);
    for (int b = 0; b < grid; ++b) {
      const int bc = s.common > 0 ? rax::share_of_block(b, s.common) : s.common;
      const int bo = b >= s.own_at ? rax::share_of_block(b - s.own_at, s.own) : s.own;
      if (bc < s.common) ++c[bc];
      if (bo < s.own) ++o[bo];
    }
    for (int x : c) TRUE(x == 1);
    for (int x : o) TRUE(x == 1);
  }
}

// A line of units: what the shares leave (whole units in their rows' state, parts in the workspace) and what the merge
// takes for a unit, which are the same steps in the same order, with no place of the workspace twice.
static void line_walk() {
  std::mt19937 g(6);
  for (int i = 0; i < 3000; ++i) {
    std::vector<int> steps;   // of each unit
    const int units = 1 + g() % 60;
    const int top = 1 + (int)(g() % 2 ? g() % 6 : g() % 300);
    for (int u = 0; u < units; ++u) steps.push_back(1 + g() % top);
    std::vector<int> at(1, 0);
    for (int x : steps) at.push_back(at.back() + x);
    const int work = at.back(), workers = 1 + (int)(g() % std::min(work, 512));
    struct Piece {
      int unit, s0, s1;
    };
    std::map<unsigned, Piece> places;
    std::vector<int> whole(units, 0);
    for (int b = 0; b < workers; ++b) {
      int x = rax::share_start(work, workers, b), u = 0;
      const int x1 = rax::share_start(work, workers, b + 1);
      while (x < x1) {
        while (x >= at[u + 1]) ++u;
        const int s0 = x - at[u], s1 = std::min(steps[u], x1 - at[u]);
        if (s0 == 0 && s1 == steps[u]) {
          ++whole[u];
        } else {
          const int first = rax::share_owner(work, workers, at[u]);
          const unsigned slot = rax::part_slot(first, b - first);
          TRUE(slot < 2u * workers && places.count(slot) == 0);
          places[slot] = Piece{u, s0, s1};
        }
        x = at[u] + s1;
      }
    }
    for (int u = 0; u < units; ++u) {
      const int first = rax::share_owner(work, workers, at[u]), parts = rax::share_owner(work, workers, at[u] + steps[u] - 1) - first + 1;
      TRUE(whole[u] == (parts == 1));
      if (parts == 1) continue;
      int s = 0;
      for (int k = 0; k < parts; ++k) {
        const unsigned slot = rax::part_slot(first, k);
        TRUE(places.count(slot) == 1 && places[slot].unit == u && places[slot].s0 == s);
        s = places[slot].s1;
      }
      TRUE(s == steps[u]);
    }
  }
}

int main() {
  select_refusals();
  fork_refusals();
  copy_refusals();
  shared_refusals();
  shape_walk();
  fork_walk();
  group_walk();
  split_walk();
  line_walk();
  std::printf("%d failures\n", failures);
  return failures != 0;
}
