// Products by group (expert), forward and backward: rows offsets[g] ...
// offsets[g + 1] of x meet the weights w[g],
//   z[m, n] = sum over k of x[m, k] w[g, n, k] + bias[g, n]
// with the epilogues, tiles and loops of linear.hip. The groups' sizes are on
// the device alone; the host knows how many rows and groups there are, and so
// how many tiles at most. Every workgroup therefore finds its own tile from the
// offsets: a lane counts the tiles of some groups, a wave adds them up. No list
// of tiles is made by a launch of its own, which would take as long as one
// token's whole product.
#define TACO_DEVICE_CODE_ONLY
#include "linear.hip"

namespace taco {

// ----------------------------------------------------------------- groups --

// First row and end of group g.
TACO_DEV int offset_at(const Groups& gr, int g) {
  const int o = gr.offsets[g];
  return o < 0 ? 0 : o > gr.rows ? gr.rows : o;
}

// Inclusive sums over a wave's lanes, by DPP: inside 16 lanes, then the last
// lane of a row of 16 to the next row, then that of 32 to the other half.
TACO_DEV unsigned lanes_scan(unsigned v) {
  auto add = [&](unsigned moved) { v += moved; };
  add((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));   // row_shr 1
  add((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));   // row_shr 2
  add((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));   // row_shr 4
  add((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));   // row_shr 8
  add((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast 15 into rows 1, 3
  add((unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast 31 into rows 2, 3
  return v;
}
TACO_DEV unsigned lane_value(unsigned v, int lane) { return (unsigned)__builtin_amdgcn_readlane((int)v, lane); }

// Tiles of 2^log rows in which the groups lie, each group beginning a new one.
struct GroupTiles {
  const Groups& gr;
  int log, per;               // groups of a lane
  unsigned mine, upto;        // tiles of this lane's groups, and of them and all before
  int lo, hi;                 // rows of this lane's group, if each has one
  TACO_DEV unsigned tiles(int first, int end) const {
    return end > first ? ((unsigned)(end - first - 1) >> log) + 1 : 0;
  }
  TACO_DEV GroupTiles(const Groups& groups, int log_rows) : gr(groups), log(log_rows) {
    const int lane = (int)threadIdx.x % kWave;
    per = (gr.count + kWave - 1) / kWave;
    mine = 0;
    lo = hi = 0;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g >= gr.count) break;
      lo = offset_at(gr, g);
      hi = offset_at(gr, g + 1);
      mine += tiles(lo, hi);
    }
    upto = lanes_scan(mine);
  }
  TACO_DEV unsigned all() const { return lane_value(upto, kWave - 1); }
};

// A group and where its tiles lie among all.
struct Group {
  int g, lo, hi;
  unsigned before, tiles;
};
// The group of tile t; false if there is none.
TACO_DEV bool group_of_tile(const GroupTiles& gt, unsigned t, Group* out) {
  const unsigned long long after = __builtin_amdgcn_ballot_w64(gt.upto > t);
  if (after == 0) return false;
  const int lane = __builtin_ctzll(after);
  out->before = lane_value(gt.upto - gt.mine, lane);
  if (gt.per == 1) {
    out->g = lane;
    out->lo = (int)lane_value((unsigned)gt.lo, lane);
    out->hi = (int)lane_value((unsigned)gt.hi, lane);
    out->tiles = gt.tiles(out->lo, out->hi);
  } else {
    const int first = lane * gt.per;
    for (int i = 0; i < gt.per; ++i) {
      out->g = first + i;
      if (out->g >= gt.gr.count) return false;
      out->lo = offset_at(gt.gr, out->g);
      out->hi = offset_at(gt.gr, out->g + 1);
      out->tiles = gt.tiles(out->lo, out->hi);
      if (t - out->before < out->tiles) break;
      out->before += out->tiles;
    }
  }
  // (offsets that go down could count more tiles than fit 32 bits)
  return t >= out->before && t - out->before < out->tiles;
}

constexpr int log2_of(int v) { return v <= 1 ? 0 : 1 + log2_of(v / 2); }

// --------------------------------------------------------------- products --

using TilesTall = Tiles<64, 128, 2, 2>;    // few rows to a group: the weights' bytes bound it
using TilesFlat = Tiles<32, 128, 2, 2>;

// Forward products (w's k contiguous), and dx = dz w (BK_). Only as many
// workgroups as the groups have tiles do anything.
template <class TL, bool BK_, bool GATED>
__global__ __launch_bounds__(TL::kThreads, 2) void k_experts(GemmArgs a, Groups gr, int64_t b_rows) {
  constexpr int BM = TL::BM, kCols = GATED ? TL::BN / 2 : TL::BN;
  const unsigned ntn = (unsigned)(a.N + kCols - 1) / kCols;
  const GroupTiles gt(gr, log2_of(BM));
  const unsigned count = gt.all() * ntn;
  if (blockIdx.x >= count) return;
  const unsigned index = xcd_ordered(blockIdx.x, count);
  Group g;
  if (!group_of_tile(gt, index / ntn, &g)) return;
  unsigned tm, tn;
  tile_of(index - g.before * ntn, g.tiles, ntn, &tm, &tn);
  Tile t;
  t.m0 = g.lo + (int64_t)tm * BM;
  t.n0 = (int)tn * kCols;
  t.N = a.N;
  t.rows = g.hi - (int)t.m0 < BM ? g.hi - (int)t.m0 : BM;
  t.cols = a.N - t.n0 < kCols ? a.N - t.n0 : kCols;
  t.K = a.K;
  t.a = a.a.p + t.m0 * a.a.ld;
  t.b = a.b.p + g.g * b_rows * a.b.ld + (BK_ ? t.n0 : t.n0 * a.b.ld);
  t.b2 = GATED ? t.b + (int64_t)a.N * a.b.ld : t.b;
  t.lda = a.a.ld;
  t.ldb = a.b.ld;
  t.part = nullptr;
  Epilogue e = a.e;
  if (!BK_ && !GATED && e.bias.p)
    e.bias.p = static_cast<char*>(e.bias.p) + g.g * e.bias.ld * (e.bias.dt == kBF16 ? 2 : 4);
  sum_tile<TL, false, BK_, GATED, Bf16>(e, t);
}

// dw[g] = the product of dz and x over the group's rows; zeros if it has none.
template <class TL>
__global__ __launch_bounds__(TL::kThreads, 2) void k_experts_dw(GemmArgs a, Groups gr) {
  constexpr int BM = TL::BM, BN = TL::BN;
  const unsigned ntm = (unsigned)((a.M + BM - 1) / BM), ntn = (unsigned)((a.N + BN - 1) / BN);
  const unsigned index = xcd_ordered(blockIdx.x, gridDim.x), per = ntm * ntn;
  const int g = (int)(index / per), lo = offset_at(gr, g), hi = offset_at(gr, g + 1);
  unsigned tm, tn;
  tile_of(index % per, ntm, ntn, &tm, &tn);
  Tile t;
  t.m0 = (int64_t)tm * BM;
  t.n0 = (int)tn * BN;
  t.N = a.N;
  t.rows = (int)(a.M - t.m0 < BM ? a.M - t.m0 : BM);
  t.cols = a.N - t.n0 < BN ? a.N - t.n0 : BN;
  t.K = hi > lo ? hi - lo : 0;
  t.a = a.a.p + lo * a.a.ld + t.m0;
  t.b = t.b2 = a.b.p + lo * a.b.ld + t.n0;
  t.lda = a.a.ld;
  t.ldb = a.b.ld;
  t.part = nullptr;
  Epilogue e = a.e;
  e.out.p = static_cast<char*>(e.out.p) + g * a.M * e.out.ld * (e.out.dt == kBF16 ? 2 : 4);
  sum_tile<TL, true, true, false, Bf16>(e, t);
}

// Few rows: of each group that has any, 16 * TM at a time.
template <int TM, bool GATED>
__global__ __launch_bounds__(kFewWaves * kWave) void k_experts_few(GemmArgs a, Groups gr, int64_t b_rows) {
  const unsigned ntn = (unsigned)(a.N + a.cols - 1) / (unsigned)a.cols;
  const GroupTiles gt(gr, 31);   // one tile to a group
  const unsigned count = gt.all() * ntn;
  if (blockIdx.x >= count) return;
  const unsigned index = xcd_ordered(blockIdx.x, count);
  Group g;
  if (!group_of_tile(gt, index / ntn, &g)) return;
  FewRows f;
  f.lda = a.a.ld * 2;
  f.ldb = a.b.ld * 2;
  f.K = a.K * 2;
  f.n0 = (int)(index - g.before * ntn) * a.cols;
  f.cols = a.N - f.n0 < a.cols ? a.N - f.n0 : a.cols;
  f.N = a.N;
  f.b = reinterpret_cast<const char*>(a.b.p + g.g * b_rows * a.b.ld);
  Epilogue e = a.e;
  if (!GATED && e.bias.p) e.bias.p = static_cast<char*>(e.bias.p) + g.g * e.bias.ld * (e.bias.dt == kBF16 ? 2 : 4);
  for (int m = g.lo; m < g.hi; m += 16 * TM) {
    f.m0 = m;
    f.rows = g.hi - m < 16 * TM ? g.hi - m : 16 * TM;
    f.a = reinterpret_cast<const char*>(a.a.p + m * a.a.ld);
    few_rows_product<TM, GATED, Bf16>(e, f);
  }
}

// ------------------------------------------- backward of activations, dbias --

// dz, and the sums over ranges of 32 rows of one group each.
constexpr int kRangeLog = 5;
template <bool GATED>
__global__ __launch_bounds__(256) void k_experts_act_back(ActBackArgs a, Groups gr, unsigned slabs, unsigned bound) {
  const GroupTiles gt(gr, kRangeLog);
  const unsigned range = blockIdx.x / slabs;
  Group g;
  if (range >= bound || !group_of_tile(gt, range, &g)) return;
  const int64_t first = g.lo + ((int64_t)(range - g.before) << kRangeLog), end = first + (1 << kRangeLog);
  act_back<GATED>(a, first, end < g.hi ? end : g.hi, range, blockIdx.x % slabs);
}

// A group's sums of those, in order; zeros for a group without rows.
__global__ __launch_bounds__(256) void k_experts_dbias(const float* partials, int N, Mat dbias, Groups gr, unsigned bound) {
  __shared__ float sums[kSumParts * kWave];
  const int g = (int)blockIdx.y;
  const GroupTiles gt(gr, kRangeLog);
  // tiles before the lane that has the group, and before it in that lane
  const int lane = g / gt.per;
  unsigned before = lane_value(gt.upto - gt.mine, lane);
  for (int i = lane * gt.per; i < g; ++i) before += gt.tiles(offset_at(gr, i), offset_at(gr, i + 1));
  const unsigned tiles = gt.tiles(offset_at(gr, g), offset_at(gr, g + 1));
  ColumnSumArgs s;
  s.in = partials + (int64_t)before * N;
  s.ld = N;
  s.second = 0;
  s.count = before <= bound && tiles <= bound - before ? (int)tiles : 0;
  s.cols = N;
  s.out[0] = {static_cast<char*>(dbias.p) + g * dbias.ld * (dbias.dt == kBF16 ? 2 : 4), N, dbias.dt};
  column_sum<4>(s, blockIdx.x, 0, sums);
}

// ----------------------------------------------------------------- launch --

// Tiles of 2^log rows that the groups can have at most.
static int64_t most_tiles(const Groups& g, int log) {
  const int64_t used = std::min(g.count, g.rows);   // groups with rows
  return (g.rows + used * ((int64_t(1) << log) - 1)) >> log;
}

bool few_rows_experts(const Groups& g, int64_t, int64_t, bool) { return g.rows <= kFewRows; }

template <class TL>
static void launch_experts_tiles(const GemmArgs& a, const Groups& g, int64_t b_rows, hipStream_t s) {
  const int cols = a.gated ? TL::BN / 2 : TL::BN;
  const dim3 grid((unsigned)(most_tiles(g, log2_of(TL::BM)) * ((a.N + cols - 1) / cols))), block(TL::kThreads);
  constexpr size_t lds = TL::kLdsBytes;
  if (a.b.by_k) hipLaunchKernelGGL((k_experts<TL, true, false>), grid, block, lds, s, a, g, b_rows);
  else if (a.gated) hipLaunchKernelGGL((k_experts<TL, false, true>), grid, block, lds, s, a, g, b_rows);
  else hipLaunchKernelGGL((k_experts<TL, false, false>), grid, block, lds, s, a, g, b_rows);
}

hipError_t launch_experts(const GemmArgs& args, const Groups& g, int64_t b_rows, hipStream_t s) {
  if (g.rows == 0) return hipSuccess;
  GemmArgs a = args;
  if (!a.b.by_k && few_rows_experts(g, a.N, a.K, a.gated)) {
    a.cols = a.gated ? 8 : 16;
    const dim3 grid((unsigned)((a.N + a.cols - 1) / a.cols) * (unsigned)std::min(g.count, g.rows));
    const dim3 block(kFewWaves * kWave);
    if (a.gated) hipLaunchKernelGGL((k_experts_few<1, true>), grid, block, 0, s, a, g, b_rows);
    else hipLaunchKernelGGL((k_experts_few<1, false>), grid, block, 0, s, a, g, b_rows);
    return hipGetLastError();
  }
  const int64_t rows = g.rows / g.count, cols = a.gated ? 2 * (int64_t)a.N : a.N;
  if (rows <= 32) launch_experts_tiles<TilesFlat>(a, g, b_rows, s);
  else if (rows <= 64) launch_experts_tiles<TilesTall>(a, g, b_rows, s);
  else if (rows >= 256 && (int64_t)g.rows * cols >= int64_t(192) << 16) launch_experts_tiles<TilesLarge>(a, g, b_rows, s);
  else launch_experts_tiles<TilesSmall>(a, g, b_rows, s);
  return hipGetLastError();
}

hipError_t launch_experts_dw(const GemmArgs& a, const Groups& g, hipStream_t s) {
  auto launch = [&](auto tiles) {
    using TL = decltype(tiles);
    const int64_t per = ((a.M + TL::BM - 1) / TL::BM) * ((a.N + TL::BN - 1) / TL::BN);
    hipLaunchKernelGGL((k_experts_dw<TL>), dim3((unsigned)(per * g.count)), dim3(TL::kThreads), TL::kLdsBytes, s, a, g);
  };
  const int64_t large = ((a.M + 255) / 256) * ((a.N + 255) / 256) * g.count;
  if (large >= 192) launch(TilesLarge());
  else launch(TilesSmall());
  return hipGetLastError();
}

int64_t experts_back_ranges(const Groups& g) { return most_tiles(g, kRangeLog); }

hipError_t launch_experts_act_back(const ActBackArgs& a, const Mat& dbias, const Groups& g, hipStream_t s) {
  const unsigned bound = (unsigned)experts_back_ranges(g), slabs = (unsigned)((a.N + 511) / 512);
  if (bound > 0) hipLaunchKernelGGL((k_experts_act_back<false>), dim3(bound * slabs), dim3(256), 0, s, a, g, slabs, bound);
  const dim3 grid((unsigned)((a.N + kWave - 1) / kWave), (unsigned)g.count);
  hipLaunchKernelGGL(k_experts_dbias, grid, dim3(256), 0, s, a.partials, a.N, dbias, g, bound);
  return hipGetLastError();
}

}  // namespace taco
