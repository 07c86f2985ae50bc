// The kernel that the grouped products' rules take for each shape on standard input (op dtype groups
// rows n k, buffers aligned to 16 bytes, 148 SMs), one line each; host only, no CUDA call.
#include <cstdio>
#include <cstring>

#include "grouped_rows.cuh"
#include "grouped_warp.cuh"
#include "grouped_wgrad.cuh"

using namespace moe;

int main() {
  char name[16], dtype[16];
  long G, rows, n, k;
  constexpr int kSms = 148;
  while (std::scanf("%15s %15s %ld %ld %ld %ld", name, dtype, &G, &rows, &n, &k) == 6) {
    const int op = !std::strcmp(name, "mm") ? kGroupedMM : !std::strcmp(name, "dgrad") ? kGroupedDgrad : kGroupedWgrad;
    const bool w = op == kGroupedWgrad, fp32 = !std::strcmp(dtype, "fp32");
    const bool tma = !fp32 && n % 8 == 0 && k % 8 == 0;
    const int parts = w ? wgrad_parts((int)G, rows, (int)n, (int)k, tma) : 1;
    const long t128 = parts * grouped_tiles(op, G, rows, n, k, 128, 128);
    const long t64 = parts * grouped_tiles(op, G, rows, n, k, 64, 64);
    if (tma && w) std::printf("tma");
    else if (tma) std::printf("tma %d", gr_tile_rows(rows, (int)G));
    else if (fp32)
      std::printf("simt %d %d", simt_tile(t128, t64, kSms),
                  simt_tile(t128, t64, kSms) > 32 && n % 4 == 0 && k % 4 == 0 ? 4 : 1);
    else std::printf("warp %d", warp_tile(t128, kSms));
    if (parts > 1) std::printf(" parts %d", parts);
    std::printf("\n");
  }
  return 0;
}
