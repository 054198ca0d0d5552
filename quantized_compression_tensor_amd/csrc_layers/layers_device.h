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
  TACO_DEV void clear() { v = u32x4{0u, 0u, 0u, 0u}; }
  TACO_DEV void opaque() { asm volatile("" : "+v"(v)); }   // the compiler forgets where the value came from
  TACO_DEV void load(const void* base, int64_t at) { __builtin_memcpy(&v, static_cast<const uint16_t*>(base) + at, 16); }
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
  TACO_DEV void clear() { lo = hi = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
  TACO_DEV void opaque() { asm volatile("" : "+v"(lo), "+v"(hi)); }
  TACO_DEV void load(const void* base, int64_t at) {
    const float* p = static_cast<const float*>(base) + at;
    __builtin_memcpy(&lo, p, 16);
    __builtin_memcpy(&hi, p + 4, 16);
  }
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
TACO_DEV void load8(const void* base, int dt, int64_t at, float* f) { load8(base, dt, at, 8, f); }
// NT: streamed past the caches, as a tensor that another kernel reads should
// be (forward norm 8192 x 5120 46.0 us cached, 39.3 streamed). A norm's waves
// write neighbouring columns of a row at about the same time, so that holds
// for rows that do not start on a line too (rows 5123 apart 46.0 and 39.9, 8192
// x 5121 55.0 and 44.0, 32768 x 1001 39.5 and 31.6; float32 rows about equal).
template <bool NT>
TACO_DEV void store16(void* p, u32x4 v) {
  typedef unsigned any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  if constexpr (NT) __builtin_nontemporal_store((any_u32x4)v, static_cast<any_u32x4*>(p));
  else *static_cast<any_u32x4*>(p) = (any_u32x4)v;
}
template <bool NT = true>
TACO_DEV void store8(void* base, int dt, int64_t at, int n, const float* f) {
  if (dt == kBF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    const u32x4 v = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7])};
    if (n >= 8) {
      store16<NT>(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    if (n >= 8) {
#pragma unroll
      for (int h = 0; h < 8; h += 4)
        store16<NT>(p + h, u32x4{__float_as_uint(f[h]), __float_as_uint(f[h + 1]), __float_as_uint(f[h + 2]),
                                 __float_as_uint(f[h + 3])});
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = f[i];
    }
  }
}
TACO_DEV void store8(void* base, int dt, int64_t at, const float* f) { store8(base, dt, at, 8, f); }
// Eight floats that stay in the caches: partial sums, read again soon.
TACO_DEV void keep8(float* p, const float* f) { store8<false>(p, kF32, 0, 8, f); }
TACO_DEV float load1(const void* base, int dt, int64_t at) {
  return dt == kBF16 ? (float)static_cast<const __bf16*>(base)[at] : static_cast<const float*>(base)[at];
}
TACO_DEV void store1(void* base, int dt, int64_t at, float f) {
  if (dt == kBF16) static_cast<__bf16*>(base)[at] = (__bf16)f;
  else static_cast<float*>(base)[at] = f;
}

// v plus the value of another lane of the same 16 (a DPP control).
template <int CTRL>
TACO_DEV float add_dpp(float v) {
  const int i = __builtin_bit_cast(int, v);
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false));
}

// Sum over the L lanes (16, 32 or 64) of an aligned group: every lane has it.
// Inside 16 lanes by DPP, which costs an add each; a wave's four sixteens
// through scalar registers.
template <int L>
TACO_DEV float lanes_sum(float v) {
  v = add_dpp<0xB1>(v);    // quad_perm 1 0 3 2
  v = add_dpp<0x4E>(v);    // quad_perm 2 3 0 1
  v = add_dpp<0x141>(v);   // row_half_mirror
  v = add_dpp<0x140>(v);   // row_mirror
  if constexpr (L == 32) v += __shfl_xor(v, 16, kWave);
  if constexpr (L == 64) {
    const int i = __builtin_bit_cast(int, v);
    auto lane = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(i, l)); };
    v = (lane(0) + lane(16)) + (lane(32) + lane(48));
  }
  return v;
}

// Column sums (ColumnSumArgs), output y: `block` takes 64 columns, every
// sixteenth row by itself, eight loads under way, so that a sum's order is the
// same for any number of waves. `sums`: 16 * 64 floats of LDS.
constexpr int kSumParts = 16;
template <int WAVES>
TACO_DEV void column_sum(const ColumnSumArgs& a, unsigned block, unsigned y, float* sums) {
  const int lane = (int)threadIdx.x % kWave, wave = wave_in_group();
  const int c = (int)block * kWave + lane;
  const Mat out = a.out[y];
  if (out.p == nullptr) return;
  const float* in = a.in + (y ? a.second : 0) + c;
#pragma unroll
  for (int part = wave; part < kSumParts; part += WAVES) {
    float t = 0.0f;
    if (c < a.cols) {
      int r = part;
      for (; r + 7 * kSumParts < a.count; r += 8 * kSumParts) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = in[(r + i * kSumParts) * a.ld];
#pragma unroll
        for (int i = 0; i < 8; ++i) t += f[i];
      }
      for (; r < a.count; r += kSumParts) t += in[r * a.ld];
    }
    sums[part * kWave + lane] = t;
  }
  __syncthreads();
  if (wave == 0 && c < a.cols) {
    float t = sums[lane];
#pragma unroll
    for (int w = 1; w < kSumParts; ++w) t += sums[w * kWave + lane];
    store1(out.p, out.dt, c, t);
  }
}

}  // namespace taco
