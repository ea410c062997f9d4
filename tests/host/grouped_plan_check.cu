// Host-side check of the grouped GEMM's work plan, compiled with nvcc against
// the kernel's own header and run on the CPU (no GPU call). For every (tiles,
// slots, kblocks, sub-tiles) tried: the units are the full tiles and then
// equal parts of the others; parts over K number at most slots in all (the
// bound of the partials' workspace and of the tile counters) and hold at least
// 4 K blocks each; parts by sub-tile appear only with two sub-tiles.
// Prints "ok" and exits 0, or prints the first violation and exits 1.
#include <cstdio>

#include "gemm.cuh"

using namespace qlora;

static int fail(const char *what, int tiles, int slots, int kb, int ntt) {
  std::printf("FAIL %s: tiles %d slots %d kblocks %d sub-tiles %d\n", what, tiles, slots, kb, ntt);
  return 1;
}

int main() {
  const int slot_list[] = {1, 2, 37, 73, 74};
  const int kb_list[] = {1, 2, 4, 7, 8, 9, 64, 172, 344};
  for (int slots : slot_list)
    for (int kb : kb_list)
      for (int ntt = 1; ntt <= 2; ++ntt)
        for (int tiles = 0; tiles <= 400; ++tiles) {
          const GroupedPlan p = plan_grouped(tiles, slots, kb, ntt);
          if (p.tiles != tiles || p.full_tiles < 0 || p.full_tiles > tiles) return fail("tiles", tiles, slots, kb, ntt);
          const int tail = tiles - p.full_tiles;
          if (p.tail_subtiles > 1 && p.tail_splits > 1) return fail("both kinds", tiles, slots, kb, ntt);
          if (p.tail_subtiles != 1 && p.tail_subtiles != ntt) return fail("sub-tiles", tiles, slots, kb, ntt);
          const int parts = p.tail_subtiles > 1 ? p.tail_subtiles : p.tail_splits;
          if (p.units != p.full_tiles + tail * parts) return fail("units", tiles, slots, kb, ntt);
          if (p.tail_splits > 1) {
            if (p.full_tiles != 0 || tiles * p.tail_splits > slots) return fail("partials bound", tiles, slots, kb, ntt);
            for (int s = 0; s < p.tail_splits; ++s) {
              const int b = static_cast<int>(static_cast<long long>(s) * kb / p.tail_splits);
              const int e = static_cast<int>(static_cast<long long>(s + 1) * kb / p.tail_splits);
              if (e - b < 4) return fail("K range", tiles, slots, kb, ntt);
            }
          }
        }
  std::printf("ok\n");
  return 0;
}
