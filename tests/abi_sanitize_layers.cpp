// The layers' argument checks and workspace sizes under AddressSanitizer and
// UndefinedBehaviorSanitizer, at the ends of the integers too. Every call is
// refused or has nothing to do, so nothing here reaches a GPU. Exit status 0
// when every result is the expected one; the sanitizers abort on the first
// error they find.
#include <math.h>
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

// Array number i, 1 GiB from the next; never read.
static taco_array at(int i, int64_t stride, int32_t dtype = TACO_BF16) {
  return taco_array{reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 30), stride, dtype, 0};
}
static const taco_array kNone = {nullptr, 0, TACO_F32, 0};
static const int64_t kSizes[] = {INT64_MIN, INT64_MIN + 1, -1, 0, INT64_MAX / 2, INT64_MAX / 2 + 1, INT64_MAX - 1,
                                 INT64_MAX};

static void sizes() {
  for (int64_t s : kSizes) {
    const int64_t three[][3] = {{s, 64, 64}, {64, s, 64}, {64, 64, s}, {s, s, s}};
    for (const auto& t : three) {
      // no rows are a size like any other, and need no workspace
      const bool fine = t[0] == 0 && t[1] > 0 && t[2] > 0;
      EXPECT(taco_linear_workspace_bytes(t[0], t[1], t[2]), 0);
      EXPECT(taco_linear_backward_workspace_bytes(t[0], t[1], t[2]) > 0, fine);
      EXPECT(taco_gated_linear_workspace_bytes(t[0], t[1], t[2]), 0);
      EXPECT(taco_gated_linear_backward_workspace_bytes(t[0], t[1], t[2]) > 0, fine);
      const taco_array a = at(0, 64), w = at(1, 64), o = at(2, 64), z = at(3, 128), p = at(4, 64), q = at(5, 64);
      if (fine) continue;
      EXPECT(taco_linear(a, w, kNone, TACO_ACT_NONE, kNone, o, kNone, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
      EXPECT(taco_gated_linear(a, w, TACO_ACT_SILU, o, z, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
      EXPECT(taco_linear_backward(o, a, w, TACO_ACT_GELU, z, p, q, kNone, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
      EXPECT(taco_gated_linear_backward(o, a, w, TACO_ACT_SILU, z, p, q, t[0], t[1], t[2], nullptr, 0, nullptr) < 0, 1);
    }
    const int64_t two[][2] = {{s, 64}, {64, s}, {s, s}};
    for (const auto& t : two) {
      EXPECT(taco_layer_norm_backward_workspace_bytes(t[0], t[1]), 0);
      if (t[0] == 0 && t[1] > 0) continue;
      EXPECT(taco_layer_norm(at(0, 64), t[0], t[1], kNone, kNone, 1e-5f, at(1, 64), nullptr, nullptr, nullptr) < 0, 1);
    }
  }
}

// Strides and addresses whose extents would pass 64 bits.
static void arrays() {
  float* const f = static_cast<float*>(at(6, 0).data);
  for (int64_t stride : {INT64_MIN, INT64_C(-1), INT64_C(0), INT64_C(63), INT64_MAX / 4, INT64_MAX}) {
    EXPECT(taco_layer_norm(at(0, stride), 4, 64, kNone, kNone, 1e-5f, at(1, 64), nullptr, nullptr, nullptr) < 0, 1);
    EXPECT(taco_layer_norm(at(0, 64), 4, 64, kNone, kNone, 1e-5f, at(1, stride), f, f + 64, nullptr) < 0, 1);
    EXPECT(taco_linear(at(0, stride), at(1, 64), kNone, TACO_ACT_NONE, kNone, at(2, 64), kNone, 4, 64, 64, nullptr, 0,
                       nullptr) < 0, 1);
    EXPECT(taco_linear(at(0, 64), at(1, 64), kNone, TACO_ACT_NONE, at(3, stride), at(2, 64), kNone, 4, 64, 64, nullptr,
                       0, nullptr) < 0, 1);
    EXPECT(taco_gated_linear(at(0, 64), at(1, 64), TACO_ACT_SILU, at(2, 64), at(3, stride), 4, 64, 64, nullptr, 0,
                             nullptr) < 0, 1);
    EXPECT(taco_linear_backward(at(0, 64), at(1, 64), at(2, 64), TACO_ACT_GELU, at(3, 64), at(4, stride), kNone, kNone,
                                4, 64, 64, at(8, 0).data, 1 << 20, nullptr) < 0, 1);
  }
  // side by side in one tensor of 128 columns, one element shared
  EXPECT(taco_layer_norm(taco_array{f, 128, TACO_F32, 0}, 4, 64, kNone, kNone, 1e-5f,
                         taco_array{f - 63, 128, TACO_F32, 0}, nullptr, nullptr, nullptr), TACO_ERR_INVALID_ARG);
  EXPECT(taco_layer_norm(at(0, 64), 4, 64, kNone, kNone, -1.0f, at(1, 64), nullptr, nullptr, nullptr),
         TACO_ERR_INVALID_ARG);
  EXPECT(taco_layer_norm(at(0, 64), 4, 64, kNone, kNone, NAN, at(1, 64), nullptr, nullptr, nullptr), TACO_ERR_INVALID_ARG);
}

// Every size that is taken has a workspace that is counted without overflow:
// the ends of the limits, and tensors of 2^35 elements.
static void limits() {
  const int64_t dim = TACO_LINEAR_MAX_DIM;
  EXPECT(taco_linear_workspace_bytes(32767, dim, dim / 32) > 0, 1);
  EXPECT(taco_linear_workspace_bytes(32769, dim, 8), 0);
  EXPECT(taco_linear_backward_workspace_bytes(32768, dim, 64) > 0, 1);
  EXPECT(taco_gated_linear_workspace_bytes(32768, dim / 2, 64) > 0, 1);
  EXPECT(taco_gated_linear_workspace_bytes(64, dim / 2 + 1, 64), 0);
  EXPECT(taco_gated_linear_backward_workspace_bytes(INT64_C(1) << 30, 16, 32) > 0, 1);
  EXPECT(taco_gated_linear_backward_workspace_bytes((INT64_C(1) << 30) + 1, 1, 1), 0);
  EXPECT(taco_layer_norm_backward_workspace_bytes(INT32_MAX, 16) > 0, 1);
  EXPECT(taco_layer_norm_backward_workspace_bytes(INT64_C(1) << 31, 1), 0);
  EXPECT(taco_layer_norm_backward_workspace_bytes(INT64_C(1) << 21, TACO_NORM_MAX_COLS), INT64_C(512) * 2 * 4 * TACO_NORM_MAX_COLS);
}

int main() {
  sizes();
  arrays();
  limits();
  if (failures) return 1;
  printf("all checks passed\n");
  return 0;
}
