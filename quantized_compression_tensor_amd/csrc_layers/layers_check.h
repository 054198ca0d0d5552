// Host code that the C ABI's files of the layers share: checks of arrays and
// sizes, workspaces, and what a call needs of one.
#pragma once

#include <initializer_list>

#include "abi_common.h"
#include "layers_internal.h"
#include "taco.h"

namespace taco {

inline int64_t elem_bytes(int dt) { return dt == TACO_BF16 ? 2 : dt == TACO_I8 ? 1 : 4; }

// An array as the kernels take it, checked against [rows, cols]; `need`: it
// may not be absent.
struct Checked {
  Mat m;
  int64_t bytes;   // from the first element to the end of the last row
  int status;
  int64_t row;     // bytes of a row's elements, and from one row to the next
  int64_t step;    // (0: one row)
};

enum Need { kOptional, kRequired };
enum Types { kAnyType, kBf16Only, kI8Only };   // any: float32 or bf16

inline bool has_type(int32_t dtype, Types types) {
  if (types == kI8Only) return dtype == TACO_I8;
  return dtype == TACO_BF16 || (types == kAnyType && dtype == TACO_F32);
}

inline Checked check_array(const taco_array& a, int64_t rows, int64_t cols, Need need, Types types = kAnyType) {
  Checked c = {{a.data, rows > 1 ? a.stride : cols, a.dtype}, 0, TACO_OK, 0, 0};
  if (a.data == nullptr) {
    if (need == kRequired && rows > 0) c.status = TACO_ERR_INVALID_ARG;
    return c;
  }
  if (a.reserved != 0) c.status = TACO_ERR_INVALID_ARG;
  else if (!has_type(a.dtype, types)) c.status = TACO_ERR_FORMAT;
  else if (rows > 1 && a.stride < cols) c.status = TACO_ERR_SHAPE;
  else if (rows > 1 && a.stride > kMaxElems / rows) c.status = TACO_ERR_INVALID_ARG;
  else if (reinterpret_cast<uintptr_t>(a.data) % (uintptr_t)elem_bytes(a.dtype) != 0) c.status = TACO_ERR_ALIGN;
  if (c.status == TACO_OK && rows > 0) {
    c.bytes = ((rows - 1) * c.m.ld + cols) * elem_bytes(a.dtype);
    c.row = cols * elem_bytes(a.dtype);
    c.step = rows > 1 ? c.m.ld * elem_bytes(a.dtype) : 0;
  }
  return c;
}

inline Checked check_vector(const taco_array& a, int64_t n, Need need) { return check_array(a, 1, n, need); }

// Float32 vectors that are not given as taco_array.
inline Checked check_floats(const float* p, int64_t n) {
  Checked c = {{const_cast<float*>(p), n, TACO_F32}, 4 * n, TACO_OK, 4 * n, 0};
  if (p == nullptr) c.bytes = 0;
  else if (reinterpret_cast<uintptr_t>(p) % 4 != 0) c.status = TACO_ERR_ALIGN;
  return c;
}

inline int first_error(std::initializer_list<const Checked*> all) {
  for (const Checked* c : all)
    if (c->status != TACO_OK) return c->status;
  return TACO_OK;
}

// Whether two arrays share a byte. Slices of columns of one tensor, which have
// one stride, lie within each other's span without sharing any where their
// columns differ.
inline bool share(const Checked& a, const Checked& b) {
  if (a.m.p == nullptr || b.m.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  if (!overlaps(a.m.p, a.bytes, b.m.p, b.bytes)) return false;
  if (a.step == 0 || a.step != b.step) return true;
  const intptr_t apart = reinterpret_cast<intptr_t>(b.m.p) - reinterpret_cast<intptr_t>(a.m.p);
  const int64_t column = (int64_t)(apart % a.step + a.step) % a.step;   // of b's first element in a's rows
  return column < a.row || column + b.row > a.step;
}

// No output may overlap an input or another output.
inline bool any_overlap(std::initializer_list<const Checked*> ins, std::initializer_list<const Checked*> outs) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Checked* i : ins)
      if (share(*i, **o)) return true;
    for (auto q = outs.begin(); q != o; ++q)
      if (share(**q, **o)) return true;
  }
  return false;
}

// A workspace of `need` bytes as an array to check for overlaps.
inline Checked check_workspace(void* ws, size_t ws_bytes, size_t need) {
  Checked c = {{need ? ws : nullptr, 0, TACO_F32}, (int64_t)need, TACO_OK, (int64_t)need, 0};
  if (need && (ws == nullptr || ws_bytes < need || !aligned16(ws))) c.status = TACO_ERR_WORKSPACE;
  return c;
}

// Sizes of a projection with `n` output columns, of as many weight rows or
// (gated) twice as many.
inline int check_linear_sizes(int64_t m, int64_t n, int64_t k, bool gated) {
  if (m < 0 || n <= 0 || k <= 0) return TACO_ERR_INVALID_ARG;
  if (n > TACO_LINEAR_MAX_DIM / (gated ? 2 : 1) || k > TACO_LINEAR_MAX_DIM) return TACO_ERR_SHAPE;
  const int64_t wide = gated ? 2 * n : n;
  if (m > (int64_t(1) << 30) || wide * k > kMaxElems || m > kMaxElems / wide || m > kMaxElems / k)
    return TACO_ERR_INVALID_ARG;
  return TACO_OK;
}

// An operand of the matrix cores.
inline Checked check_operand(const taco_array& a, int64_t rows, int64_t cols, Types type = kBf16Only) {
  Checked c = check_array(a, rows, cols, kRequired, type);
  if (c.status == TACO_OK && c.m.ld > TACO_LINEAR_MAX_STRIDE) c.status = TACO_ERR_SHAPE;
  return c;
}

inline int check_act(int32_t act) { return act >= TACO_ACT_NONE && act <= TACO_ACT_RELU ? TACO_OK : TACO_ERR_FORMAT; }

inline Operand operand(const Checked& c, bool by_k) { return Operand{static_cast<const uint16_t*>(c.m.p), c.m.ld, by_k}; }

constexpr Mat kAbsent = {nullptr, 0, TACO_F32};

inline int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Whether the tiles can be loaded from where a matrix lies: rows on 16 bytes,
// whole eights in each.
inline bool in_place(const Mat& m, int64_t cols) {
  return aligned16(m.p) && m.ld % 8 == 0 && cols % 8 == 0;
}

// Elements from one row to the next in the workspace: whole 128-byte lines,
// except in narrow matrices. A tile's step is one line of each row then, not
// parts of two (8171 x 507 x 6647 122 us, with rows on 16 bytes 144).
inline int64_t packed_ld(int64_t cols) { return up(cols, cols < 64 ? 8 : 64); }

// Takes parts of a workspace, each a multiple of 256 bytes; without a base it
// only counts.
struct Space {
  char* base;
  size_t used;
  void* take(size_t bytes) {
    void* p = base ? base + used : nullptr;
    used += (size_t)up((int64_t)bytes, 256);
    return p;
  }
};

// What a pass over a call is for: the workspace that arrays of any alignment
// would need with all outputs asked for, the workspace that this call needs,
// or its launches.
enum Pass { kSizeOfAny, kSize, kRun };

// A bf16 matrix [rows, cols] as an operand: in place, or packed into `space`
// (added to `pack`).
inline Operand packed(const Mat& m, int64_t rows, int64_t cols, bool by_k, bool whole, Space* space, PackArgs* pack) {
  if (whole) return Operand{static_cast<const uint16_t*>(m.p), m.ld, by_k};
  const int64_t ld = packed_ld(cols);
  uint16_t* dst = static_cast<uint16_t*>(space->take((size_t)(rows * ld) * 2));
  pack->m[pack->count++] = {m, rows, cols, dst, ld};
  return Operand{dst, ld, by_k};
}

template <class Call>
size_t space_of(const Call& c, Pass what) {
  Space s = {nullptr, 0};
  (void)c.pass(what, &s, nullptr);
  return s.used;
}

template <class Call>
int run(const Call& c, void* ws, hipStream_t stream) {
  Space s = {static_cast<char*>(ws), 0};
  clear_stale_error();
  return hip_status(c.pass(kRun, &s, stream));
}

}  // namespace taco
