// The layers' part of the C ABI: validation and dispatch, all of it host code;
// every check runs before any work is enqueued.
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "abi_common.h"
#include "layers_internal.h"
#include "taco.h"

namespace {

using namespace taco;

int64_t elem_bytes(int dt) { return dt == TACO_BF16 ? 2 : 4; }

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
enum Types { kAnyType, kBf16Only };

Checked check_array(const taco_array& a, int64_t rows, int64_t cols, Need need, Types types = kAnyType) {
  Checked c = {{a.data, rows > 1 ? a.stride : cols, a.dtype}, 0, TACO_OK, 0, 0};
  if (a.data == nullptr) {
    if (need == kRequired && rows > 0) c.status = TACO_ERR_INVALID_ARG;
    return c;
  }
  if (a.reserved != 0) c.status = TACO_ERR_INVALID_ARG;
  else if (a.dtype != TACO_F32 && a.dtype != TACO_BF16) c.status = TACO_ERR_FORMAT;
  else if (types == kBf16Only && a.dtype != TACO_BF16) c.status = TACO_ERR_FORMAT;
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

Checked check_vector(const taco_array& a, int64_t n, Need need) { return check_array(a, 1, n, need); }

// Float32 vectors that are not given as taco_array.
Checked check_floats(const float* p, int64_t n) {
  Checked c = {{const_cast<float*>(p), n, TACO_F32}, 4 * n, TACO_OK, 4 * n, 0};
  if (p == nullptr) c.bytes = 0;
  else if (reinterpret_cast<uintptr_t>(p) % 4 != 0) c.status = TACO_ERR_ALIGN;
  return c;
}

int first_error(std::initializer_list<const Checked*> all) {
  for (const Checked* c : all)
    if (c->status != TACO_OK) return c->status;
  return TACO_OK;
}

// Whether two arrays share a byte. Slices of columns of one tensor, which have
// one stride, lie within each other's span without sharing any where their
// columns differ.
bool share(const Checked& a, const Checked& b) {
  if (a.m.p == nullptr || b.m.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  if (!overlaps(a.m.p, a.bytes, b.m.p, b.bytes)) return false;
  if (a.step == 0 || a.step != b.step) return true;
  const intptr_t apart = reinterpret_cast<intptr_t>(b.m.p) - reinterpret_cast<intptr_t>(a.m.p);
  const int64_t column = (int64_t)(apart % a.step + a.step) % a.step;   // of b's first element in a's rows
  return column < a.row || column + b.row > a.step;
}

// No output may overlap an input or another output.
bool any_overlap(std::initializer_list<const Checked*> ins, std::initializer_list<const Checked*> outs) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    for (const Checked* i : ins)
      if (share(*i, **o)) return true;
    for (auto q = outs.begin(); q != o; ++q)
      if (share(**q, **o)) return true;
  }
  return false;
}

// A workspace of `need` bytes as an array to check for overlaps.
Checked check_workspace(void* ws, size_t ws_bytes, size_t need) {
  Checked c = {{need ? ws : nullptr, 0, TACO_F32}, (int64_t)need, TACO_OK, (int64_t)need, 0};
  if (need && (ws == nullptr || ws_bytes < need || !aligned16(ws))) c.status = TACO_ERR_WORKSPACE;
  return c;
}

int check_norm_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return TACO_ERR_INVALID_ARG;
  if (cols > TACO_NORM_MAX_COLS) return TACO_ERR_SHAPE;
  if (rows > kMaxElems / cols || rows > INT32_MAX) return TACO_ERR_INVALID_ARG;
  return TACO_OK;
}

// Sizes of a projection with `n` output columns, of as many weight rows or
// (gated) twice as many.
int check_linear_sizes(int64_t m, int64_t n, int64_t k, bool gated) {
  if (m < 0 || n <= 0 || k <= 0) return TACO_ERR_INVALID_ARG;
  if (n > TACO_LINEAR_MAX_DIM / (gated ? 2 : 1) || k > TACO_LINEAR_MAX_DIM) return TACO_ERR_SHAPE;
  const int64_t wide = gated ? 2 * n : n;
  if (m > (int64_t(1) << 30) || wide * k > kMaxElems || m > kMaxElems / wide || m > kMaxElems / k)
    return TACO_ERR_INVALID_ARG;
  return TACO_OK;
}

// An operand of the matrix cores.
Checked check_operand(const taco_array& a, int64_t rows, int64_t cols) {
  Checked c = check_array(a, rows, cols, kRequired, kBf16Only);
  if (c.status == TACO_OK && c.m.ld > TACO_LINEAR_MAX_STRIDE) c.status = TACO_ERR_SHAPE;
  return c;
}

int check_act(int32_t act) { return act >= TACO_ACT_NONE && act <= TACO_ACT_RELU ? TACO_OK : TACO_ERR_FORMAT; }

Operand operand(const Checked& c, bool by_k) { return Operand{static_cast<const uint16_t*>(c.m.p), c.m.ld, by_k}; }

constexpr Mat kAbsent = {nullptr, 0, TACO_F32};

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Whether the tiles can be loaded from where a matrix lies: rows on 16 bytes,
// whole eights in each.
bool in_place(const Mat& m, int64_t cols) {
  return aligned16(m.p) && m.ld % 8 == 0 && cols % 8 == 0;
}

// Elements from one row to the next in the workspace: whole 128-byte lines,
// except in narrow matrices. A tile's step is one line of each row then, not
// parts of two (8171 x 507 x 6647 122 us, with rows on 16 bytes 144).
int64_t packed_ld(int64_t cols) { return up(cols, cols < 64 ? 8 : 64); }

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
Operand packed(const Mat& m, int64_t rows, int64_t cols, bool by_k, bool whole, Space* space, PackArgs* pack) {
  if (whole) return Operand{static_cast<const uint16_t*>(m.p), m.ld, by_k};
  const int64_t ld = packed_ld(cols);
  uint16_t* dst = static_cast<uint16_t*>(space->take((size_t)(rows * ld) * 2));
  pack->m[pack->count++] = {m, rows, cols, dst, ld};
  return Operand{dst, ld, by_k};
}

// A call of either kind of projection: what it needs of the workspace, and
// its launches. `wide`: rows of w.
struct Forward {
  Checked x, w;
  Epilogue e;
  bool gated;
  int64_t m, n, k;
  hipError_t pass(Pass what, Space* space, hipStream_t stream) const {
    const bool worst = what == kSizeOfAny;
    const int64_t wide = gated ? 2 * n : n;
    const bool few = few_rows(m, n, k, gated);
    PackArgs pack = {};
    GemmArgs g = {};
    g.a = packed(x.m, m, k, false, few || (!worst && in_place(x.m, k)), space, &pack);
    g.b = packed(w.m, wide, k, false, few || (!worst && in_place(w.m, k)), space, &pack);
    g.M = m; g.N = (int)n; g.K = k; g.gated = gated; g.e = e;
    void* partials = space->take(few ? 0 : gemm_partial_bytes(m, n, k, gated));
    if (what != kRun) return hipSuccess;
    if (pack.count > 0) {
      const hipError_t err = launch_pack(pack, stream);
      if (err != hipSuccess) return err;
    }
    return launch_gemm(g, partials, stream);
  }
};

struct Backward {
  Checked dout, x, w, z, dx, dw, db;
  int act;
  bool gated;
  int64_t m, n, k;
  hipError_t pass(Pass what, Space* space, hipStream_t stream) const {
    const bool worst = what == kSizeOfAny;
    const int64_t wide = gated ? 2 * n : n, ld_dz = packed_ld(wide);
    const bool want_dx = worst || (dx.m.p && m > 0), want_dw = worst || dw.m.p, want_db = !gated && (worst || db.m.p);
    // dz is dout itself where there is no activation and the tiles can take it
    const bool own_dz = worst || gated || act != TACO_ACT_NONE || ((want_dx || want_dw) && !in_place(dout.m, n));
    PackArgs pack = {};
    ActBackArgs b = {};
    b.dout = dout.m; b.z = z.m; b.M = m; b.N = (int)n; b.act = act; b.gated = gated; b.ld_dz = ld_dz;
    Operand dz = {static_cast<const uint16_t*>(dout.m.p), dout.m.ld, false};
    if (own_dz) {
      b.dz = static_cast<uint16_t*>(space->take((size_t)(m * ld_dz) * 2));
      dz = Operand{b.dz, ld_dz, false};
    }
    Operand ox = {}, ow = {};
    if (want_dw) ox = packed(x.m, m, k, true, !worst && in_place(x.m, k), space, &pack);
    if (want_dx) ow = packed(w.m, wide, k, true, !worst && in_place(w.m, k), space, &pack);
    // used in turn
    const size_t dx_bytes = want_dx ? gemm_partial_bytes(m, k, wide, false) : 0;
    const size_t dw_bytes = want_dw ? gemm_partial_bytes(wide, k, m, false) : 0;
    const size_t db_bytes = want_db ? (size_t)act_back_groups(m) * (size_t)n * sizeof(float) : 0;
    const size_t both_bytes = want_dx && want_dw ? gemm_pair_partial_bytes(m, wide, k) : 0;
    void* rest = space->take(std::max({dx_bytes, dw_bytes, both_bytes}));
    if (want_db) b.partials = static_cast<float*>(space->take(db_bytes));
    if (what != kRun) return hipSuccess;
    const ColumnSumArgs sum = {b.partials, n, 0, act_back_groups(m), (int)n, {want_db ? db.m : kAbsent, kAbsent}};
    hipError_t err = hipSuccess;
    if (own_dz || want_db) err = launch_act_back(b, pack, stream);
    else if (pack.count > 0) err = launch_pack(pack, stream);
    if (err != hipSuccess) return err;
    GemmArgs gx = {}, gw = {};
    gx.a = dz; gx.b = ow; gx.M = m; gx.N = (int)k; gx.K = wide; gx.e.out = dx.m;
    dz.by_k = true;
    gw.a = dz; gw.b = ox; gw.M = wide; gw.N = (int)k; gw.K = m; gw.e.out = dw.m;
    if (want_dx && want_dw) return launch_gemm_pair(gx, gw, sum, rest, stream);
    launch_column_sum(sum, stream);
    if (want_dx) return launch_gemm(gx, rest, stream);
    if (want_dw) return launch_gemm(gw, rest, stream);
    return hipGetLastError();
  }
};

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

size_t forward_bytes(bool gated, int64_t m, int64_t n, int64_t k) {
  if (check_linear_sizes(m, n, k, gated) != TACO_OK) return 0;
  Forward f = {};
  f.gated = gated; f.m = m; f.n = n; f.k = k;
  return space_of(f, kSizeOfAny);
}
size_t backward_bytes(bool gated, int64_t m, int64_t n, int64_t k) {
  if (check_linear_sizes(m, n, k, gated) != TACO_OK) return 0;
  Backward b = {};
  b.gated = gated; b.m = m; b.n = n; b.k = k;
  return space_of(b, kSizeOfAny);
}

}  // namespace

extern "C" {

int taco_layer_norm(taco_array x, int64_t rows, int64_t cols, taco_array weight, taco_array bias, float eps,
                    taco_array y, float* mean, float* rstd, hipStream_t stream) {
  int st = check_norm_sizes(rows, cols);
  if (st != TACO_OK) return st;
  if (!(eps >= 0.0f) || isinf(eps)) return TACO_ERR_INVALID_ARG;
  const Checked cx = check_array(x, rows, cols, kRequired), cy = check_array(y, rows, cols, kRequired);
  const Checked cw = check_vector(weight, cols, kOptional), cb = check_vector(bias, cols, kOptional);
  const Checked cm = check_floats(mean, rows), cr = check_floats(rstd, rows);
  st = first_error({&cx, &cy, &cw, &cb, &cm, &cr});
  if (st != TACO_OK) return st;
  if (any_overlap({&cx, &cw, &cb}, {&cy, &cm, &cr})) return TACO_ERR_INVALID_ARG;
  if (rows == 0) return TACO_OK;
  const NormArgs a = {cx.m, cw.m, cb.m, cy.m, rows, (int)cols, eps, mean, rstd, 0};
  clear_stale_error();
  return hip_status(launch_norm(a, stream));
}

size_t taco_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (check_norm_sizes(rows, cols) != TACO_OK) return 0;
  return (size_t)norm_back_groups(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

int taco_layer_norm_backward(taco_array dy, taco_array x, int64_t rows, int64_t cols, taco_array weight,
                             const float* mean, const float* rstd, taco_array dx, taco_array dweight,
                             taco_array dbias, void* workspace, size_t ws_bytes, hipStream_t stream) {
  int st = check_norm_sizes(rows, cols);
  if (st != TACO_OK) return st;
  const Checked cdy = check_array(dy, rows, cols, kRequired), cx = check_array(x, rows, cols, kRequired);
  const Checked cw = check_vector(weight, cols, kOptional), cdx = check_array(dx, rows, cols, kOptional);
  const Checked cdw = check_vector(dweight, cols, kOptional), cdb = check_vector(dbias, cols, kOptional);
  const Checked cm = check_floats(mean, rows), cr = check_floats(rstd, rows);
  st = first_error({&cdy, &cx, &cw, &cdx, &cdw, &cdb, &cm, &cr});
  if (st != TACO_OK) return st;
  if (rows > 0 && (mean == nullptr || rstd == nullptr)) return TACO_ERR_INVALID_ARG;
  const bool sums = dweight.data != nullptr || dbias.data != nullptr;
  if (rows > 0 && !sums && dx.data == nullptr) return TACO_ERR_INVALID_ARG;
  const Checked cws =
      check_workspace(workspace, ws_bytes, sums ? taco_layer_norm_backward_workspace_bytes(rows, cols) : 0);
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cdy, &cx, &cw, &cm, &cr}, {&cdx, &cdw, &cdb, &cws})) return TACO_ERR_INVALID_ARG;
  if (rows == 0 && !sums) return TACO_OK;
  const NormBackArgs a = {cdy.m, cx.m, cw.m, cdx.m, cdw.m, cdb.m, rows, (int)cols, mean, rstd,
                          static_cast<float*>(cws.m.p), 0};
  clear_stale_error();
  return hip_status(launch_norm_back(a, stream));
}

size_t taco_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) { return forward_bytes(false, M, N, K); }

int taco_linear(taco_array x, taco_array w, taco_array bias, int32_t act, taco_array residual, taco_array out,
                taco_array preact, int64_t M, int64_t N, int64_t K, void* workspace, size_t ws_bytes,
                hipStream_t stream) {
  int st = check_linear_sizes(M, N, K, false);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const Checked cx = check_operand(x, M, K), cw = check_operand(w, N, K), cb = check_vector(bias, N, kOptional);
  const Checked cr = check_array(residual, M, N, kOptional), co = check_array(out, M, N, kRequired);
  const Checked cz = check_array(preact, M, N, kOptional);
  st = first_error({&cx, &cw, &cb, &cr, &co, &cz});
  if (st != TACO_OK) return st;
  const Forward f = {cx, cw, {cb.m, cr.m, cz.m, co.m, act}, false, M, N, K};
  const Checked cws = check_workspace(workspace, ws_bytes, space_of(f, kSize));
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cx, &cw, &cb, &cr}, {&co, &cz, &cws})) return TACO_ERR_INVALID_ARG;
  return M == 0 ? TACO_OK : run(f, cws.m.p, stream);
}

size_t taco_gated_linear_workspace_bytes(int64_t M, int64_t F, int64_t K) { return forward_bytes(true, M, F, K); }

int taco_gated_linear(taco_array x, taco_array w, int32_t act, taco_array out, taco_array preact, int64_t M,
                      int64_t F, int64_t K, void* workspace, size_t ws_bytes, hipStream_t stream) {
  int st = check_linear_sizes(M, F, K, true);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const Checked cx = check_operand(x, M, K), cw = check_operand(w, 2 * F, K);
  const Checked co = check_array(out, M, F, kRequired), cz = check_array(preact, M, 2 * F, kOptional);
  st = first_error({&cx, &cw, &co, &cz});
  if (st != TACO_OK) return st;
  const Forward f = {cx, cw, {kAbsent, kAbsent, cz.m, co.m, act}, true, M, F, K};
  const Checked cws = check_workspace(workspace, ws_bytes, space_of(f, kSize));
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cx, &cw}, {&co, &cz, &cws})) return TACO_ERR_INVALID_ARG;
  return M == 0 ? TACO_OK : run(f, cws.m.p, stream);
}

size_t taco_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) { return backward_bytes(false, M, N, K); }

int taco_linear_backward(taco_array dout, taco_array x, taco_array w, int32_t act, taco_array preact, taco_array dx,
                         taco_array dw, taco_array dbias, int64_t M, int64_t N, int64_t K, void* workspace,
                         size_t ws_bytes, hipStream_t stream) {
  int st = check_linear_sizes(M, N, K, false);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const Checked cd = check_operand(dout, M, N), cx = check_operand(x, M, K), cw = check_operand(w, N, K);
  const Checked cz = check_array(preact, M, N, act == TACO_ACT_NONE ? kOptional : kRequired);
  const Checked cdx = check_array(dx, M, K, kOptional), cdw = check_array(dw, N, K, kOptional);
  const Checked cdb = check_vector(dbias, N, kOptional);
  st = first_error({&cd, &cx, &cw, &cz, &cdx, &cdw, &cdb});
  if (st != TACO_OK) return st;
  if (M > 0 && !dx.data && !dw.data && !dbias.data) return TACO_ERR_INVALID_ARG;
  const Backward b = {cd, cx, cw, cz, cdx, cdw, cdb, act, false, M, N, K};
  const Checked cws = check_workspace(workspace, ws_bytes, space_of(b, kSize));
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cd, &cx, &cw, &cz}, {&cdx, &cdw, &cdb, &cws})) return TACO_ERR_INVALID_ARG;
  if (M == 0 && !dw.data && !dbias.data) return TACO_OK;
  return run(b, cws.m.p, stream);
}

size_t taco_gated_linear_backward_workspace_bytes(int64_t M, int64_t F, int64_t K) {
  return backward_bytes(true, M, F, K);
}

int taco_gated_linear_backward(taco_array dout, taco_array x, taco_array w, int32_t act, taco_array preact,
                               taco_array dx, taco_array dw, int64_t M, int64_t F, int64_t K, void* workspace,
                               size_t ws_bytes, hipStream_t stream) {
  int st = check_linear_sizes(M, F, K, true);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const Checked cd = check_operand(dout, M, F), cx = check_operand(x, M, K), cw = check_operand(w, 2 * F, K);
  const Checked cz = check_array(preact, M, 2 * F, kRequired);
  const Checked cdx = check_array(dx, M, K, kOptional), cdw = check_array(dw, 2 * F, K, kOptional);
  st = first_error({&cd, &cx, &cw, &cz, &cdx, &cdw});
  if (st != TACO_OK) return st;
  if (M > 0 && !dx.data && !dw.data) return TACO_ERR_INVALID_ARG;
  const Backward b = {cd, cx, cw, cz, cdx, cdw, {kAbsent, 0, TACO_OK, 0, 0}, act, true, M, F, K};
  const Checked cws = check_workspace(workspace, ws_bytes, space_of(b, kSize));
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cd, &cx, &cw, &cz}, {&cdx, &cdw, &cws})) return TACO_ERR_INVALID_ARG;
  if (M == 0 && !dw.data) return TACO_OK;
  return run(b, cws.m.p, stream);
}

}  // extern "C"
