// For each line "groups M N K" of the standard input, of a forward product by
// group: its tile's rows, tiles at most, parts of K, threads of its launch and
// those of the ranges of its gradient's sums; and the same for dx ("N" columns,
// "K" rows of weights). Host code only; needs no GPU.
#include <stdio.h>

#include "../quantized_compression_tensor_amd/csrc_layers/experts.hip"

namespace taco {
void launch_column_sum(const ColumnSumArgs&, hipStream_t) {}   // never called
}  // namespace taco

int main() {
  long long groups, m, n, k;
  while (scanf("%lld %lld %lld %lld", &groups, &m, &n, &k) == 4) {
    const taco::Groups g = {nullptr, (int)groups, (int)m};
    for (int dx = 0; dx < 2; ++dx) {
      const taco::ExpertsPlan p = dx ? taco::dx_plan(g, n, k, true) : taco::experts_plan(g, n, k, false, false);
      int height = 0, threads = 0;
      taco::with_tiles(p.shape, [&](auto tiles) {
        height = decltype(tiles)::BM;
        threads = decltype(tiles)::kThreads;
      });
      const long long ranges = taco::experts_back_ranges(g) * ((n + 511) / 512) * 256;
      printf("%d %lld %u %lld %lld\n", height, (long long)p.tiles, p.parts, (long long)p.tiles * p.parts * threads, ranges);
    }
  }
  return 0;
}
