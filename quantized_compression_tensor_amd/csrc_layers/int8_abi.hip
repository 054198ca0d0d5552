// The C ABI of the projections in 8-bit integers: validation and dispatch, all
// of it host code; every check runs before any work is enqueued.
#include <algorithm>

#include "layers_check.h"

namespace {

using namespace taco;

int check_int8_sizes(int64_t m, int64_t n, int64_t k, bool gated) {
  const int st = check_linear_sizes(m, n, k, gated);
  return st == TACO_OK && k > TACO_INT8_MAX_K ? TACO_ERR_SHAPE : st;
}

// A matrix of codes as the tiles' operand, in pairs of codes: in place where
// its rows lie on 16 bytes and hold whole sixteens, or copied so into `space`,
// each row on a 128-byte line except in narrow matrices (as packed()).
Operand packed_codes(const Mat& m, int64_t rows, int64_t cols, bool whole, Space* space, PackArgs* pack) {
  if (whole) return Operand{static_cast<const uint16_t*>(m.p), m.ld / 2, false};
  const int64_t ld = up(cols, cols < 128 ? 16 : 128);
  uint16_t* dst = static_cast<uint16_t*>(space->take((size_t)(rows * ld)));
  pack->m[pack->count++] = {m, rows, cols, dst, ld};
  return Operand{dst, ld / 2, false};
}
bool codes_in_place(const Mat& m, int64_t cols) { return aligned16(m.p) && m.ld % 16 == 0 && cols % 16 == 0; }

struct Int8Call {
  Checked x, w;
  Epilogue e;
  bool gated;
  int64_t m, n, k;
  hipError_t pass(Pass what, Space* space, hipStream_t stream) const {
    const bool worst = what == kSizeOfAny;
    GemmArgs g = {};
    g.M = m; g.N = (int)n; g.gated = gated; g.e = e;
    const bool few = few_rows_int8(m, n, k, gated), direct = !few && direct_int8(m, n, k, gated);
    const bool aligned = !worst && codes_in_place(x.m, k) && codes_in_place(w.m, k);
    if (few || (direct && !aligned)) {
      g.K = k;
      g.a = Operand{static_cast<const uint16_t*>(x.m.p), x.m.ld, false};
      g.b = Operand{static_cast<const uint16_t*>(w.m.p), w.m.ld, false};
      // (arrays of any alignment: aligned ones, too)
      const size_t own = direct ? direct_int8_bytes(m, n, k, gated) : 0;
      const size_t tiles = worst && !few ? gemm_partial_bytes(m, n, up(k, 16) / 2, gated) : 0;
      void* partials = space->take(std::max(own, tiles));
      return what == kRun ? launch_gemm_int8(few ? kInt8Few : kInt8Direct, g, partials, stream) : hipSuccess;
    }
    PackArgs pack = {};
    g.K = up(k, 16) / 2;
    g.a = packed_codes(x.m, m, k, !worst && codes_in_place(x.m, k), space, &pack);
    g.b = packed_codes(w.m, gated ? 2 * n : n, k, !worst && codes_in_place(w.m, k), space, &pack);
    void* partials = space->take(gemm_partial_bytes(m, n, g.K, gated));
    if (what != kRun) return hipSuccess;
    if (pack.count > 0) {
      const hipError_t err = launch_pack_int8(pack, stream);
      if (err != hipSuccess) return err;
    }
    return launch_gemm_int8(kInt8Tiles, g, partials, stream);
  }
};

size_t int8_bytes(bool gated, int64_t m, int64_t n, int64_t k) {
  if (check_int8_sizes(m, n, k, gated) != TACO_OK) return 0;
  Int8Call c = {};
  c.gated = gated; c.m = m; c.n = n; c.k = k;
  return space_of(c, kSizeOfAny);
}

int int8_call(bool gated, const taco_array& x, const float* x_scale, const taco_array& w, const float* w_scale,
              const taco_array& bias, int32_t act, const taco_array& residual, const taco_array& out, int64_t M,
              int64_t N, int64_t K, void* workspace, size_t ws_bytes, hipStream_t stream) {
  int st = check_int8_sizes(M, N, K, gated);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const int64_t wide = gated ? 2 * N : N;
  const Checked cx = check_operand(x, M, K, kI8Only), cw = check_operand(w, wide, K, kI8Only);
  const Checked cxs = check_floats(x_scale, M), cws = check_floats(w_scale, wide);
  const Checked cb = check_vector(bias, N, kOptional), cr = check_array(residual, M, N, kOptional);
  const Checked co = check_array(out, M, N, kRequired);
  st = first_error({&cx, &cw, &cxs, &cws, &cb, &cr, &co});
  if (st != TACO_OK) return st;
  if (w_scale == nullptr || (M > 0 && x_scale == nullptr)) return TACO_ERR_INVALID_ARG;
  const Int8Call c = {cx, cw, {cb.m, cr.m, kAbsent, co.m, act, x_scale, w_scale}, gated, M, N, K};
  const Checked cspace = check_workspace(workspace, ws_bytes, space_of(c, kSize));
  if (cspace.status != TACO_OK) return cspace.status;
  if (any_overlap({&cx, &cw, &cxs, &cws, &cb, &cr}, {&co, &cspace})) return TACO_ERR_INVALID_ARG;
  return M == 0 ? TACO_OK : run(c, cspace.m.p, stream);
}

}  // namespace

extern "C" {

int taco_quantize_rows(taco_array x, int64_t rows, int64_t cols, taco_array q, float* scale, hipStream_t stream) {
  if (rows < 0 || cols <= 0) return TACO_ERR_INVALID_ARG;
  if (cols > TACO_LINEAR_MAX_DIM) return TACO_ERR_SHAPE;
  if (rows > kMaxElems / cols) return TACO_ERR_INVALID_ARG;
  const Checked cx = check_array(x, rows, cols, kRequired), cq = check_array(q, rows, cols, kRequired, kI8Only);
  const Checked cs = check_floats(scale, rows);
  const int st = first_error({&cx, &cq, &cs});
  if (st != TACO_OK) return st;
  if (rows > 0 && scale == nullptr) return TACO_ERR_INVALID_ARG;
  if (any_overlap({&cx}, {&cq, &cs})) return TACO_ERR_INVALID_ARG;
  if (rows == 0) return TACO_OK;
  clear_stale_error();
  return hip_status(launch_quantize(QuantizeArgs{cx.m, cq.m, rows, cols, scale}, stream));
}

size_t taco_linear_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) { return int8_bytes(false, M, N, K); }

int taco_linear_int8(taco_array x, const float* x_scale, taco_array w, const float* w_scale, taco_array bias, int32_t act,
                     taco_array residual, taco_array out, int64_t M, int64_t N, int64_t K, void* workspace,
                     size_t ws_bytes, hipStream_t stream) {
  return int8_call(false, x, x_scale, w, w_scale, bias, act, residual, out, M, N, K, workspace, ws_bytes, stream);
}

size_t taco_gated_linear_int8_workspace_bytes(int64_t M, int64_t F, int64_t K) { return int8_bytes(true, M, F, K); }

int taco_gated_linear_int8(taco_array x, const float* x_scale, taco_array w, const float* w_scale, int32_t act,
                           taco_array out, int64_t M, int64_t F, int64_t K, void* workspace, size_t ws_bytes,
                           hipStream_t stream) {
  const taco_array none = {nullptr, 0, TACO_F32, 0};
  return int8_call(true, x, x_scale, w, w_scale, none, act, none, out, M, F, K, workspace, ws_bytes, stream);
}

}  // extern "C"
