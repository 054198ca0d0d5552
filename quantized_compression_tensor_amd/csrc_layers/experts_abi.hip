// The C ABI of the projections by group: validation and dispatch, all of it
// host code; every check runs before any work is enqueued. What the offsets on
// the device hold is not known here: the kernels keep to the arrays whatever it
// is.
#include <algorithm>

#include "layers_check.h"

namespace {

using namespace taco;

int check_group_sizes(int32_t groups, int64_t m, int64_t n, int64_t k, bool gated) {
  const int st = check_linear_sizes(m, n, k, gated);
  if (st != TACO_OK) return st;
  if (groups <= 0) return TACO_ERR_INVALID_ARG;
  if (groups > TACO_MAX_GROUPS) return TACO_ERR_SHAPE;
  return groups * (gated ? 2 * n : n) > kMaxElems / k ? TACO_ERR_INVALID_ARG : TACO_OK;
}

Checked check_offsets(const int32_t* p, int32_t groups) {
  const int64_t bytes = 4 * ((int64_t)groups + 1);
  Checked c = {{const_cast<int32_t*>(p), groups + 1, TACO_F32}, bytes, TACO_OK, bytes, 0};
  if (p == nullptr) c.status = TACO_ERR_INVALID_ARG;
  else if (reinterpret_cast<uintptr_t>(p) % 4 != 0) c.status = TACO_ERR_ALIGN;
  return c;
}

struct GroupedForward {
  Checked x, w;
  Epilogue e;
  Groups groups;
  bool gated;
  int64_t m, n, k;
  hipError_t pass(Pass what, Space* space, hipStream_t stream) const {
    const bool worst = what == kSizeOfAny;
    const int64_t wide = gated ? 2 * n : n;
    const bool any = few_rows_experts(groups, n, k, gated) || direct_experts(groups, wide);   // as they are
    PackArgs pack = {};
    GemmArgs g = {};
    g.a = packed(x.m, m, k, false, any || (!worst && in_place(x.m, k)), space, &pack);
    g.b = packed(w.m, groups.count * wide, k, false, any || (!worst && in_place(w.m, k)), space, &pack);
    g.direct = any && !(in_place(x.m, k) && in_place(w.m, k));
    g.M = m; g.N = (int)n; g.K = k; g.gated = gated; g.e = e;
    size_t sums = 0;
    if (!few_rows_experts(groups, n, k, gated)) {
      if (worst || g.direct) sums = any ? experts_partial_bytes(groups, n, k, gated, true) : 0;
      if (worst || !g.direct) sums = std::max(sums, experts_partial_bytes(groups, n, k, gated, false));
    }
    void* partials = space->take(sums);
    if (what != kRun) return hipSuccess;
    if (pack.count > 0) {
      const hipError_t err = launch_pack(pack, stream);
      if (err != hipSuccess) return err;
    }
    return launch_experts(g, groups, wide, partials, stream);
  }
};

struct GroupedBackward {
  Checked dout, x, w, z, dx, dw, db;
  int act;
  Groups groups;
  bool gated;
  int64_t m, n, k;
  hipError_t pass(Pass what, Space* space, hipStream_t stream) const {
    const bool worst = what == kSizeOfAny;
    const int64_t wide = gated ? 2 * n : n, ld_dz = packed_ld(wide);
    const bool want_dx = worst || (dx.m.p && m > 0), want_dw = worst || dw.m.p, want_db = !gated && (worst || db.m.p);
    // dz is dout itself where there is no activation and the tiles can take it
    const bool own_dz =
        (want_dx || want_dw) && (worst || gated || act != TACO_ACT_NONE || !in_place(dout.m, n));
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
    const bool direct = direct_experts(groups, k);
    if (want_dx) ow = packed(w.m, groups.count * wide, k, true, direct || (!worst && in_place(w.m, k)), space, &pack);
    if (want_db) b.partials = static_cast<float*>(space->take((size_t)(experts_back_ranges(groups) * n) * sizeof(float)));
    void* partials = space->take(want_dx ? experts_back_bytes(groups, k, wide) : 0);
    if (what != kRun) return hipSuccess;
    hipError_t err = hipSuccess;
    if (want_db) {
      err = launch_experts_act_back(b, groups, stream);
      if (err == hipSuccess && pack.count > 0) err = launch_pack(pack, stream);
    } else if (own_dz) {
      err = launch_act_back(b, pack, stream);
    } else if (pack.count > 0) {
      err = launch_pack(pack, stream);
    }
    if (err != hipSuccess) return err;
    GemmArgs gx = {}, gw = {};
    gx.a = dz; gx.b = ow; gx.M = m; gx.N = (int)k; gx.K = wide; gx.e.out = dx.m;
    gx.direct = direct && !in_place(w.m, k);
    dz.by_k = true;
    gw.a = dz; gw.b = ox; gw.M = wide; gw.N = (int)k; gw.K = m; gw.e.out = dw.m;
    return launch_experts_back(want_dx ? &gx : nullptr, want_dw ? &gw : nullptr, b.partials, n, want_db ? db.m : kAbsent,
                               groups, wide, partials, stream);
  }
};

size_t forward_bytes(bool gated, int32_t groups, int64_t m, int64_t n, int64_t k) {
  if (check_group_sizes(groups, m, n, k, gated) != TACO_OK) return 0;
  GroupedForward f = {};
  f.groups = {nullptr, groups, (int)m};
  f.gated = gated; f.m = m; f.n = n; f.k = k;
  return space_of(f, kSizeOfAny);
}
size_t backward_bytes(bool gated, int32_t groups, int64_t m, int64_t n, int64_t k) {
  if (check_group_sizes(groups, m, n, k, gated) != TACO_OK) return 0;
  GroupedBackward b = {};
  b.groups = {nullptr, groups, (int)m};
  b.gated = gated; b.m = m; b.n = n; b.k = k;
  return space_of(b, kSizeOfAny);
}

int forward_call(bool gated, const taco_array& x, const taco_array& w, const taco_array& bias, int32_t act,
                 const int32_t* offsets, int32_t groups, const taco_array& out, const taco_array& preact, int64_t M,
                 int64_t N, int64_t K, void* workspace, size_t ws_bytes, hipStream_t stream) {
  int st = check_group_sizes(groups, M, N, K, gated);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const int64_t wide = gated ? 2 * N : N;
  const Checked cx = check_operand(x, M, K), cw = check_operand(w, groups * wide, K);
  const Checked cb = check_array(bias, groups, N, kOptional), cf = check_offsets(offsets, groups);
  const Checked co = check_array(out, M, N, kRequired), cz = check_array(preact, M, wide, kOptional);
  st = first_error({&cx, &cw, &cb, &cf, &co, &cz});
  if (st != TACO_OK) return st;
  const GroupedForward f = {cx, cw, {cb.m, kAbsent, cz.m, co.m, act}, {offsets, groups, (int)M}, gated, M, N, K};
  const Checked cws = check_workspace(workspace, ws_bytes, space_of(f, kSize));
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cx, &cw, &cb, &cf}, {&co, &cz, &cws})) return TACO_ERR_INVALID_ARG;
  return M == 0 ? TACO_OK : run(f, cws.m.p, stream);
}

int backward_call(bool gated, const taco_array& dout, const taco_array& x, const taco_array& w, int32_t act,
                  const taco_array& preact, const int32_t* offsets, int32_t groups, const taco_array& dx,
                  const taco_array& dw, const taco_array& dbias, int64_t M, int64_t N, int64_t K, void* workspace,
                  size_t ws_bytes, hipStream_t stream) {
  int st = check_group_sizes(groups, M, N, K, gated);
  if (st != TACO_OK) return st;
  st = check_act(act);
  if (st != TACO_OK) return st;
  const int64_t wide = gated ? 2 * N : N;
  const Checked cd = check_operand(dout, M, N), cx = check_operand(x, M, K), cw = check_operand(w, groups * wide, K);
  const Checked cz = check_array(preact, M, wide, gated || act != TACO_ACT_NONE ? kRequired : kOptional);
  const Checked cf = check_offsets(offsets, groups), cdx = check_array(dx, M, K, kOptional);
  const Checked cdw = check_array(dw, groups * wide, K, kOptional), cdb = check_array(dbias, groups, N, kOptional);
  st = first_error({&cd, &cx, &cw, &cz, &cf, &cdx, &cdw, &cdb});
  if (st != TACO_OK) return st;
  if (M > 0 && !dx.data && !dw.data && !dbias.data) return TACO_ERR_INVALID_ARG;
  const GroupedBackward b = {cd, cx, cw, cz, cdx, cdw, cdb, act, {offsets, groups, (int)M}, gated, M, N, K};
  const Checked cws = check_workspace(workspace, ws_bytes, space_of(b, kSize));
  if (cws.status != TACO_OK) return cws.status;
  if (any_overlap({&cd, &cx, &cw, &cz, &cf}, {&cdx, &cdw, &cdb, &cws})) return TACO_ERR_INVALID_ARG;
  if (M == 0 && !dw.data && !dbias.data) return TACO_OK;
  return run(b, cws.m.p, stream);
}

constexpr taco_array kNone = {nullptr, 0, TACO_F32, 0};

}  // namespace

extern "C" {

size_t taco_grouped_linear_workspace_bytes(int32_t groups, int64_t M, int64_t N, int64_t K) {
  return forward_bytes(false, groups, M, N, K);
}

int taco_grouped_linear(taco_array x, taco_array w, taco_array bias, int32_t act, const int32_t* offsets, int32_t groups,
                        taco_array out, taco_array preact, int64_t M, int64_t N, int64_t K, void* workspace,
                        size_t ws_bytes, hipStream_t stream) {
  return forward_call(false, x, w, bias, act, offsets, groups, out, preact, M, N, K, workspace, ws_bytes, stream);
}

size_t taco_grouped_linear_backward_workspace_bytes(int32_t groups, int64_t M, int64_t N, int64_t K) {
  return backward_bytes(false, groups, M, N, K);
}

int taco_grouped_linear_backward(taco_array dout, taco_array x, taco_array w, int32_t act, taco_array preact,
                                 const int32_t* offsets, int32_t groups, taco_array dx, taco_array dw,
                                 taco_array dbias, int64_t M, int64_t N, int64_t K, void* workspace, size_t ws_bytes,
                                 hipStream_t stream) {
  return backward_call(false, dout, x, w, act, preact, offsets, groups, dx, dw, dbias, M, N, K, workspace, ws_bytes,
                       stream);
}

size_t taco_grouped_gated_linear_workspace_bytes(int32_t groups, int64_t M, int64_t F, int64_t K) {
  return forward_bytes(true, groups, M, F, K);
}

int taco_grouped_gated_linear(taco_array x, taco_array w, int32_t act, const int32_t* offsets, int32_t groups,
                              taco_array out, taco_array preact, int64_t M, int64_t F, int64_t K, void* workspace,
                              size_t ws_bytes, hipStream_t stream) {
  return forward_call(true, x, w, kNone, act, offsets, groups, out, preact, M, F, K, workspace, ws_bytes, stream);
}

size_t taco_grouped_gated_linear_backward_workspace_bytes(int32_t groups, int64_t M, int64_t F, int64_t K) {
  return backward_bytes(true, groups, M, F, K);
}

int taco_grouped_gated_linear_backward(taco_array dout, taco_array x, taco_array w, int32_t act, taco_array preact,
                                       const int32_t* offsets, int32_t groups, taco_array dx, taco_array dw, int64_t M,
                                       int64_t F, int64_t K, void* workspace, size_t ws_bytes, hipStream_t stream) {
  return backward_call(true, dout, x, w, act, preact, offsets, groups, dx, dw, kNone, M, F, K, workspace, ws_bytes,
                       stream);
}

}  // extern "C"
