// Host-side rules of the grouped products, checked without a GPU (the program makes no CUDA
// call).  Exit status 0 = every rule holds; the first violations are printed.
#include <algorithm>
#include <cstdio>

#include "grouped_rows.cuh"
#include "grouped_warp.cuh"
#include "grouped_wgrad.cuh"

using namespace moe;

static int fails = 0;
#define CHECK(cond, ...)                                  \
  do {                                                    \
    if (!(cond)) {                                        \
      if (fails++ < 10) {                                 \
        std::printf("FAIL %s: ", #cond);                  \
        std::printf(__VA_ARGS__);                         \
        std::printf("\n");                                \
      }                                                   \
    }                                                     \
  } while (0)

int main() {
  const size_t smem = 227 * 1024;   // opt-in limit of a CTA, static and dynamic together
  // rings inside shared memory, beside the tables; whole swizzle atoms; two accumulators in TMEM
  for (int rt : {64, 256}) {
    CHECK(gr_stages(rt) >= 2 && gr_stages(rt) <= kGrMaxStages, "tile_rows=%d", rt);
    CHECK((size_t)gr_stages(rt) * gr_stage_bytes(rt) <= kGrRingBytes, "tile_rows=%d", rt);
    CHECK(gr_stage_bytes(rt) % 1024 == 0 && (rt / 2) * 128 % 1024 == 0, "tile_rows=%d", rt);
    CHECK(2 * rt <= 512 && rt % 32 == 0, "tile_rows=%d", rt);
  }
  CHECK(kGrSmemBytes + sizeof(GroupTable) + 512 <= smem, "rows kernel: %zu", kGrSmemBytes + sizeof(GroupTable));
  CHECK(kGwSmemBytes + sizeof(WgradTable) + 512 <= smem, "wgrad kernel: %zu", kGwSmemBytes + sizeof(WgradTable));
  CHECK(sizeof(GroupTable) + 4 * (WarpTile<false, 128>::kSize * 2 + WarpTile<true, 128>::kSize * 2) <= 48 * 1024 * 2,
        "warp kernel");
  // barriers in the control block: rows 2 S + 5, wgrad 4 S + 5 + 4 slots, and the two words
  CHECK((2 * kGrMaxStages + 5) * 8 + 8 <= 1024 && (4 * kGwStages + 5 + 4 * kGwSlots) * 8 + 8 <= 1024, "control");
  // rows per tile: both kinds are chosen, by the rows per expert
  CHECK(gr_tile_rows(384, 64) == 64 && gr_tile_rows(2048, 64) == 64 && gr_tile_rows(2049, 64) == 256, "rule");

  // splits: at least one; all parts together within the slots; parts of at least `least` rows on
  // average
  for (int G : {1, 2, 7, 64, 1024})
    for (long rows = 1; rows < (1l << 30); rows = rows * 3 + 1)
      for (long tiles = G; tiles < 4096; tiles = tiles * 2 + G)
        for (int slots : {74, 592})
          for (int least : {512, 1024}) {
            const int s = wgrad_splits(rows, G, tiles, slots, least);
            CHECK(s >= 1 && s <= 256, "s=%d", s);
            CHECK(s == 1 || (long)s * tiles <= slots, "G=%d rows=%ld tiles=%ld s=%d", G, rows, tiles, s);
            CHECK(s == 1 || rows / G >= (long)s * least, "G=%d rows=%ld tiles=%ld s=%d", G, rows, tiles, s);
          }
  // the parts of an expert's rows: consecutive, none missing, none twice; whole MMA steps but the
  // last; empty ones behind it
  for (int splits = 1; splits <= 256; splits = splits * 2 + 1)
    for (int rows = 0; rows < 70000; rows += rows < 600 ? 1 : 997) {
      int at = 1000;
      for (int s = 0; s < splits; ++s) {
        int r0 = 1000, n = rows;
        split_rows(r0, n, splits, s);
        CHECK(r0 == at && n >= 0, "splits=%d rows=%d s=%d r0=%d n=%d", splits, rows, s, r0, n);
        at = r0 + n;
        CHECK(n % 16 == 0 || at == 1000 + rows, "splits=%d rows=%d s=%d n=%d", splits, rows, s, n);
      }
      CHECK(at == 1000 + rows, "splits=%d rows=%d ends at %d", splits, rows, at - 1000);
    }
  if (fails) return 1;
  std::printf("all operator rules hold\n");
  return 0;
}
