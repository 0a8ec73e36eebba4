// Which workgroup of the attention takes which share, walked on the host (kv_index.h) for devices of every
// number of compute units.  Test infrastructure only.
#include <cstdio>
#include <vector>

#include "kv_index.h"

int main() {
  int failures = 0;
  for (int cus = 1; cus <= 320; ++cus) {
    const int most = rax::attention_workers(cus);
    if (most < 1 || most > 512 || most % (2 * rax::kDies)) {
      std::printf("%d compute units: %d workgroups\n", cus, most);
      ++failures;
      continue;
    }
    for (int grid : {most, most / 2, 4 * most, 2 * most})   // heads to 128 dims and above, one-wave workgroups
      for (int workers = 1; workers <= grid; workers += workers < 40 ? 1 : 7) {
        std::vector<int> taken(workers + 1);
        for (int block = 0; block < grid; ++block) ++taken[rax::share_of_block(block, workers)];
        for (int b = 0; b < workers; ++b)
          if (taken[b] != 1) {
            std::printf("grid %d, %d shares: share %d taken %d times\n", grid, workers, b, taken[b]);
            ++failures;
          }
        for (int die = 0, per = (workers + rax::kDies - 1) / rax::kDies; die < rax::kDies; ++die) {   // a run each
          int n = 0;
          for (int block = die; block < grid; block += rax::kDies)
            if (rax::share_of_block(block, workers) < workers) failures += rax::share_of_block(block, workers) != die * per + n++;
          failures += n > per;
        }
      }
  }
  std::printf("%d failures\n", failures);
  return failures != 0;
}
