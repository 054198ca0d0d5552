// Device helpers shared by the layers' kernels.
#pragma once

#include "device_common.h"
#include "layers_internal.h"

namespace taco {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Two floats -> two bf16 in one dword (the hardware conversion, nearest-even).
TACO_DEV uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v.x = (__bf16)a;
  v.y = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// Eight consecutive elements as they lie in memory. Rows may start at any
// element, so the loads and stores promise no alignment beyond it (the
// hardware takes such 16-byte accesses in one instruction); a row's last
// elements, fewer than eight, go one by one and nothing past them is touched.
template <int DT>
struct Oct;
template <>
struct Oct<kBF16> {
  u32x4 v;
  TACO_DEV void load(const void* base, int64_t at, int n) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (n >= 8) {
      __builtin_memcpy(&v, p, 16);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) w[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
      v = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
  TACO_DEV void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(v[i]);
      f[2 * i + 1] = bf16_hi(v[i]);
    }
  }
};
template <>
struct Oct<kF32> {
  f32x4 lo, hi;
  TACO_DEV void load(const void* base, int64_t at, int n) {
    const float* p = static_cast<const float*>(base) + at;
    if (n >= 8) {
      __builtin_memcpy(&lo, p, 16);
      __builtin_memcpy(&hi, p + 4, 16);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.0f;
      lo = f32x4{f[0], f[1], f[2], f[3]};
      hi = f32x4{f[4], f[5], f[6], f[7]};
    }
  }
  TACO_DEV void get(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = lo[i];
      f[4 + i] = hi[i];
    }
  }
};

// The same with the element type known at run time (wave-uniform).
TACO_DEV void load8(const void* base, int dt, int64_t at, int n, float* f) {
  if (dt == kBF16) {
    Oct<kBF16> o;
    o.load(base, at, n);
    o.get(f);
  } else {
    Oct<kF32> o;
    o.load(base, at, n);
    o.get(f);
  }
}
TACO_DEV void store8(void* base, int dt, int64_t at, int n, const float* f) {
  if (dt == kBF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    const u32x4 v = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    if (n >= 8) {
      __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    if (n >= 8) {
      __builtin_memcpy(p, f, 16);
      __builtin_memcpy(p + 4, f + 4, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = f[i];
    }
  }
}
TACO_DEV void store1(void* base, int dt, int64_t at, float f) {
  if (dt == kBF16) static_cast<__bf16*>(base)[at] = (__bf16)f;
  else static_cast<float*>(base)[at] = f;
}

// Sum over the L lanes (a power of two) of an aligned group: every lane has it.
template <int L>
TACO_DEV float lanes_sum(float v) {
#pragma unroll
  for (int m = 1; m < L; m *= 2) v += __shfl_xor(v, m, kWave);
  return v;
}

}  // namespace taco
