// Refusals of lora_beam_select where an output lies inside the logits, on the CPU with hip_stubs.cpp.  Test infrastructure only.
#include <cstdio>

#include "beam.h"
#include "raxlora.h"
#include "shared.h"

extern int g_launches;
namespace rax {
hipError_t launch_beam_select(const BeamArgs&, hipStream_t, const KTimer&) { ++g_launches; return hipSuccess; }
hipError_t launch_page_fork(const PageForkArgs&, hipStream_t, const KTimer&) { return hipSuccess; }
hipError_t launch_page_copy(const PageCopyArgs&, hipStream_t, const KTimer&) { return hipSuccess; }
}  // namespace rax

static int failures = 0;
static void expect(int line, int got, int want) {
  if (got != want) {
    std::printf("line %d: %d, want %d (%s)\n", line, got, want, lora_last_error());
    ++failures;
  }
}
#define EXPECT(call, want) expect(__LINE__, (call), (want))

int main() {
  alignas(16) static char all[1 << 16];   // logits in the middle
  alignas(16) static int32_t v[3][64];
  alignas(16) static float fl[2][64];
  char* const logits = all + (1 << 15);
  lora_beams* b = nullptr;
  EXPECT(lora_beams_create(&b, 0, 4, 4, 100, 3), LORA_OK);
  for (const lora_dtype dt : {LORA_BF16, LORA_F32}) {
    const int size = dt == LORA_F32 ? 4 : 2, ld = 120;
    for (int requests = 1; requests <= 4; ++requests) {
      const int used = ((requests * 4 - 1) * ld + 100) * size, out = requests * 3 * 4;
      for (int which = 0; which < 4; ++which) {
        const auto call = [&](char* at) {
          int32_t* const p = reinterpret_cast<int32_t*>(at);
          return lora_beam_select(b, logits, ld, dt, fl[0], nullptr, -1, nullptr, requests, which == 0 ? p : v[0], which == 1 ? p : v[1],
                                  which == 2 ? reinterpret_cast<float*>(at) : fl[1], which == 3 ? p : v[2], nullptr);
        };
        const int before = g_launches;
        for (char* at : {logits, logits + 40, logits + used - 4, logits - out + 4}) EXPECT(call(at), LORA_ERR_INVALID_ARG);
        EXPECT(g_launches, before);
        for (char* at : {logits - out, logits + used}) EXPECT(call(at), LORA_OK);   // side by side
        EXPECT(g_launches, before + 2);
      }
    }
  }
  EXPECT(lora_beams_destroy(b), LORA_OK);
  std::printf("%d failures\n", failures);
  return failures != 0;
}
