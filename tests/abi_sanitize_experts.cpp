// As abi_sanitize_layers.cpp, for the projections by group and in 8 bits: argument
// checks and workspace sizes at the ends of the integers. Every call is refused
// or has nothing to do, so nothing here reaches a GPU.
#include <stdint.h>
#include <stdio.h>

#include "taco.h"

static int failures = 0;

#define EXPECT(expr, want)                                                                    \
  do {                                                                                        \
    const long long got_ = (long long)(expr);                                                 \
    if (got_ != (long long)(want)) {                                                          \
      fprintf(stderr, "line %d: %s = %lld, expected %lld\n", __LINE__, #expr, got_, (long long)(want)); \
      ++failures;                                                                             \
    }                                                                                         \
  } while (0)

static taco_array at(int i, int64_t stride, int32_t dtype = TACO_BF16) {
  return taco_array{reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 30), stride, dtype, 0};
}
static float* floats(int i) { return static_cast<float*>(at(i, 0).data); }
static const int32_t* offsets() { return static_cast<const int32_t*>(at(9, 0).data); }
static const taco_array kNone = {nullptr, 0, TACO_F32, 0};
static const int64_t kSizes[] = {INT64_MIN, INT64_MIN + 1, -1, INT64_MAX / 2, INT64_MAX / 2 + 1, INT64_MAX - 1, INT64_MAX};

static void sizes() {
  for (int64_t s : kSizes) {
    const int64_t three[][3] = {{s, 64, 64}, {64, s, 64}, {64, 64, s}, {s, s, s}};
    for (const auto& t : three) {
      EXPECT(taco_linear_int8_workspace_bytes(t[0], t[1], t[2]), 0);
      EXPECT(taco_gated_linear_int8_workspace_bytes(t[0], t[1], t[2]), 0);
      const taco_array x = at(0, 64, TACO_I8), w = at(1, 64, TACO_I8), o = at(2, 64);
      EXPECT(taco_linear_int8(x, floats(3), w, floats(4), kNone, 0, kNone, o, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
      EXPECT(taco_gated_linear_int8(x, floats(3), w, floats(4), 0, o, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
      for (int32_t g : {INT32_MIN, 0, 1, 64, 1024, 1025, INT32_MAX}) {
        EXPECT(taco_grouped_linear_workspace_bytes(g, t[0], t[1], t[2]), 0);
        EXPECT(taco_grouped_linear_backward_workspace_bytes(g, t[0], t[1], t[2]), 0);
        EXPECT(taco_grouped_gated_linear_workspace_bytes(g, t[0], t[1], t[2]), 0);
        EXPECT(taco_grouped_gated_linear_backward_workspace_bytes(g, t[0], t[1], t[2]), 0);
        const taco_array bx = at(0, 64), bw = at(1, 64), z = at(5, 128), p = at(6, 64), q = at(7, 64);
        EXPECT(taco_grouped_linear(bx, bw, kNone, 0, offsets(), g, o, kNone, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
        EXPECT(taco_grouped_gated_linear(bx, bw, 2, offsets(), g, o, z, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
        EXPECT(taco_grouped_linear_backward(o, bx, bw, 1, z, offsets(), g, p, q, kNone, t[0], t[1], t[2], nullptr, 0,
                                            nullptr) < 0, 1);
        EXPECT(taco_grouped_gated_linear_backward(o, bx, bw, 2, z, offsets(), g, p, q, t[0], t[1], t[2], nullptr, 0,
                                                  nullptr) < 0, 1);
      }
    }
    const int64_t two[][2] = {{s, 64}, {64, s}, {s, s}};
    for (const auto& t : two)
      EXPECT(taco_quantize_rows(at(0, 64), t[0], t[1], at(1, 64, TACO_I8), floats(2), nullptr) < 0, 1);
  }
}

static void arrays() {
  for (int64_t stride : {INT64_MIN, INT64_C(-1), INT64_C(0), INT64_C(63), INT64_MAX / 4, INT64_MAX}) {
    EXPECT(taco_quantize_rows(at(0, stride), 4, 64, at(1, 64, TACO_I8), floats(2), nullptr) < 0, 1);
    EXPECT(taco_quantize_rows(at(0, 64), 4, 64, at(1, stride, TACO_I8), floats(2), nullptr) < 0, 1);
    EXPECT(taco_linear_int8(at(0, stride, TACO_I8), floats(3), at(1, 64, TACO_I8), floats(4), kNone, 0, kNone, at(2, 64),
                            4, 64, 64, nullptr, 0, nullptr) < 0, 1);
    EXPECT(taco_gated_linear_int8(at(0, 64, TACO_I8), floats(3), at(1, stride, TACO_I8), floats(4), 0, at(2, 64), 4, 64,
                                  64, nullptr, 0, nullptr) < 0, 1);
    EXPECT(taco_grouped_linear(at(0, 64), at(1, stride), kNone, 0, offsets(), 3, at(2, 64), kNone, 4, 64, 64, nullptr, 0,
                               nullptr) < 0, 1);
    EXPECT(taco_grouped_linear(at(0, 64), at(1, 64), at(3, stride), 0, offsets(), 3, at(2, 64), kNone, 4, 64, 64, nullptr,
                               0, nullptr) < 0, 1);
    EXPECT(taco_grouped_linear_backward(at(0, 64), at(1, 64), at(2, 64), 1, at(3, 64), offsets(), 3, kNone, at(4, stride),
                                        kNone, 4, 64, 64, at(8, 0).data, 1 << 28, nullptr) < 0, 1);
  }
}

static void limits() {
  const int64_t dim = TACO_LINEAR_MAX_DIM;
  EXPECT(taco_linear_int8_workspace_bytes(32768, dim, 64) > 0, 1);
  EXPECT(taco_linear_int8_workspace_bytes(INT64_C(1) << 18, 4096, TACO_INT8_MAX_K) > 0, 1);
  EXPECT(taco_linear_int8_workspace_bytes(64, 64, TACO_INT8_MAX_K + 1), 0);
  EXPECT(taco_gated_linear_int8_workspace_bytes(INT64_C(1) << 30, 16, 32) > 0, 1);
  EXPECT(taco_gated_linear_int8_workspace_bytes((INT64_C(1) << 30) + 1, 1, 1), 0);
  EXPECT(taco_grouped_linear_workspace_bytes(1024, 32768, dim, 32), 0);   // taken from where it lies
  EXPECT(taco_grouped_linear_workspace_bytes(32, INT64_C(1) << 25, 1024, 1024) > 0, 1);
  EXPECT(taco_grouped_linear_workspace_bytes(1024, 32768, dim, 33), 0);
  EXPECT(taco_grouped_gated_linear_workspace_bytes(1024, 32768, dim / 2, 32), 0);
  EXPECT(taco_grouped_gated_linear_workspace_bytes(32, INT64_C(1) << 25, 512, 1024) > 0, 1);
  EXPECT(taco_grouped_linear_backward_workspace_bytes(1024, INT64_C(1) << 30, 32, 32) > 0, 1);
  EXPECT(taco_grouped_gated_linear_backward_workspace_bytes(1024, INT64_C(1) << 30, 16, 32) > 0, 1);
  EXPECT(taco_grouped_linear_backward_workspace_bytes(1, 4, 8, 8) > 0, 1);
}

int main() {
  sizes();
  arrays();
  limits();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
