// Prints how the grouped GEMM cuts its work, from the kernel's own function
// compiled for the host (no GPU call): for each "tiles slots kblocks
// sub-tiles" given as arguments, one line "units full_tiles splits subtiles".
#include <cstdio>
#include <cstdlib>

#include "gemm.cuh"

int main(int argc, char **argv) {
  for (int i = 1; i + 3 < argc; i += 4) {
    const qlora::GroupedPlan p =
        qlora::plan_grouped(std::atoi(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2]), std::atoi(argv[i + 3]));
    std::printf("%d %d %d %d\n", p.units, p.full_tiles, p.tail_splits, p.tail_subtiles);
  }
  return 0;
}
