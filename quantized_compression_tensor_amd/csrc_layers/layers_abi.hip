// The layers' part of the C ABI: validation and dispatch, all of it host code;
// every check runs before any work is enqueued.
#include <math.h>

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
};

enum Need { kOptional, kRequired };
enum Types { kAnyType, kBf16Only };

Checked check_array(const taco_array& a, int64_t rows, int64_t cols, Need need, Types types = kAnyType) {
  Checked c = {{a.data, a.stride, a.dtype}, 0, TACO_OK};
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
  if (rows <= 1) c.m.ld = cols;
  if (c.status == TACO_OK && rows > 0) c.bytes = ((rows - 1) * c.m.ld + cols) * elem_bytes(a.dtype);
  return c;
}

Checked check_vector(const taco_array& a, int64_t n, Need need) { return check_array(a, 1, n, need); }

// Float32 vectors that are not given as taco_array.
Checked check_floats(const float* p, int64_t n) {
  Checked c = {{const_cast<float*>(p), n, TACO_F32}, 4 * n, TACO_OK};
  if (p == nullptr) c.bytes = 0;
  else if (reinterpret_cast<uintptr_t>(p) % 4 != 0) c.status = TACO_ERR_ALIGN;
  return c;
}

int first_error(std::initializer_list<const Checked*> all) {
  for (const Checked* c : all)
    if (c->status != TACO_OK) return c->status;
  return TACO_OK;
}

// No output may overlap an input or another output.
bool any_overlap(std::initializer_list<const Checked*> ins, std::initializer_list<const Checked*> outs) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if ((*o)->m.p == nullptr || (*o)->bytes == 0) continue;
    for (const Checked* i : ins)
      if (i->m.p && i->bytes && overlaps(i->m.p, i->bytes, (*o)->m.p, (*o)->bytes)) return true;
    for (auto q = outs.begin(); q != o; ++q)
      if ((*q)->m.p && (*q)->bytes && overlaps((*q)->m.p, (*q)->bytes, (*o)->m.p, (*o)->bytes)) return true;
  }
  return false;
}

// A workspace of `need` bytes as an array to check for overlaps.
Checked check_workspace(void* ws, size_t ws_bytes, size_t need) {
  Checked c = {{need ? ws : nullptr, 0, TACO_F32}, (int64_t)need, TACO_OK};
  if (need && (ws == nullptr || ws_bytes < need || !aligned16(ws))) c.status = TACO_ERR_WORKSPACE;
  return c;
}

int check_norm_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return TACO_ERR_INVALID_ARG;
  if (cols > TACO_NORM_MAX_COLS) return TACO_ERR_SHAPE;
  if (rows > kMaxElems / cols || rows > INT32_MAX) return TACO_ERR_INVALID_ARG;
  return TACO_OK;
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
  const NormArgs a = {cx.m, cw.m, cb.m, cy.m, rows, (int)cols, eps, mean, rstd};
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
  if (!sums && dx.data == nullptr) return TACO_ERR_INVALID_ARG;
  const Checked cws =
      check_workspace(workspace, ws_bytes, sums ? taco_layer_norm_backward_workspace_bytes(rows, cols) : 0);
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cdy, &cx, &cw, &cm, &cr}, {&cdx, &cdw, &cdb, &cws})) return TACO_ERR_INVALID_ARG;
  if (rows == 0 && !sums) return TACO_OK;
  const NormBackArgs a = {cdy.m, cx.m, cw.m, cdx.m, cdw.m, cdb.m, rows, (int)cols, mean, rstd,
                          static_cast<float*>(cws.m.p)};
  clear_stale_error();
  return hip_status(launch_norm_back(a, stream));
}

}  // extern "C"
