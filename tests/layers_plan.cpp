// Prints the plan of products: for each line "M N K gated" of the standard
// input, "large whole rest parts" as csrc_layers/linear.hip chooses them, and
// for "M N K pair" whether a projection's gradients are one launch. Host code
// only; needs no GPU.
#include <stdio.h>
#include <string.h>

#include "../quantized_compression_tensor_amd/csrc_layers/linear.hip"

namespace taco {
void launch_column_sum(const ColumnSumArgs&, hipStream_t) {}   // never called
}  // namespace taco

int main() {
  long long m, n, k;
  char what[16];
  while (scanf("%lld %lld %lld %15s", &m, &n, &k, what) == 4) {
    if (strcmp(what, "pair") == 0) {
      printf("%d\n", (int)taco::pair_plan_of(m, n, k).together);
    } else {
      const taco::Plan p = taco::plan_of(m, n, k, strcmp(what, "gated") == 0);
      printf("%d %u %u %u\n", (int)p.large, p.whole, p.rest, p.parts);
    }
  }
  return 0;
}
