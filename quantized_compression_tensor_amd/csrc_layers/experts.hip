// Products by group (expert), forward and backward: rows offsets[g] ...
// offsets[g + 1] of x meet the weights w[g],
//   z[m, n] = sum over k of x[m, k] w[g, n, k] + bias[g, n]
// with the epilogues, tiles and loops of linear.hip. The groups' sizes are on
// the device alone; the host knows how many rows and groups there are, and so
// how many tiles at most. Every workgroup therefore finds its own tile from the
// offsets: a lane counts the tiles of some groups, a wave adds them up. No list
// of tiles is made by a launch of its own, which would take as long as one
// token's whole product.
// Few rows to a group: bound by the weights' bytes (one token of eight experts out
// of 64, gated 2 x 1024 x 2048, 15.2 us, 67 MB at 4.4 TB/s); many: by the matrix cores
// (8192 rows over 8 groups of 2 x 4096 x 4096, both projections kept, 510 to 535 us,
// 1050 TFLOP/s of the rows' own products; profiled 518 us, busy 0.60 of the time at
// 1.89 GHz. The rows left in tiles cost 0.05 of the work, a tile's first loads and
// its stores, beside which nothing runs, 0.1).
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

// Which tiles of 2^log rows are counted of a group, whose first row begins a
// new one: all, those that it fills, or, for the rows left, ones of 2^rest_log.
enum Count { kAllTiles, kFullTiles, kRestTiles };
TACO_DEV unsigned tiles_of_rows(Count what, int rows, int log, int rest_log) {
  if (rows <= 0) return 0;
  const unsigned full = (unsigned)rows >> log, left = (unsigned)rows - (full << log);
  if (what == kAllTiles) return full + (left != 0);
  return what == kFullTiles ? full : left == 0 ? 0 : ((left - 1) >> rest_log) + 1;
}

// The groups' tiles, counted: each lane has some groups.
template <Count WHAT>
struct GroupTiles {
  const Groups& gr;
  int log, rest_log, per;     // groups of a lane
  unsigned mine, upto;        // tiles of this lane's groups, and of them and all before
  int lo, hi;                 // rows of this lane's group, if each has one
  TACO_DEV unsigned tiles(int first, int end) const { return tiles_of_rows(WHAT, end - first, log, rest_log); }
  TACO_DEV GroupTiles(const Groups& groups, int log_rows, int log_rest = 0)
      : gr(groups), log(log_rows), rest_log(log_rest) {
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

// A group and where its counted tiles lie among all.
struct Group {
  int g, lo, hi;
  unsigned before, tiles;
};
// The group of tile t; false if there is none.
template <Count WHAT>
TACO_DEV bool group_of_tile(const GroupTiles<WHAT>& gt, unsigned t, Group* out) {
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

using TilesHalf = Tiles<128, 256, 2, 4>;
// What takes the rows that do not fill a tile.
template <class TL>
struct RestOf;
template <>
struct RestOf<TilesLarge> { using Type = TilesHalf; };
template <>
struct RestOf<TilesSmall> { using Type = TilesTall; };
template <>
struct RestOf<TilesTall> { using Type = TilesFlat; };
template <>
struct RestOf<TilesFlat> { using Type = TilesFlat; };

// A tile of the groups' output rows: those that are full come first, then those
// of the rows left, half as high, which waste less and even out the last round.
struct RowTile {
  Group g;
  int m0;
  unsigned tn;
  bool full;
};
// Where tile `index` lies, of `full` and `rest`; false if there is none. Full
// tiles are in one contiguous range for each XCD (index from xcd_ordered()).
TACO_DEV bool locate(const GroupTiles<kFullTiles>& full, const GroupTiles<kRestTiles>& rest, unsigned ntn,
                     unsigned index, RowTile* t) {
  const unsigned count = full.all() * ntn;
  unsigned tm;
  t->full = index < count;
  if (t->full) {
    if (!group_of_tile(full, index / ntn, &t->g)) return false;
    tile_of(index - t->g.before * ntn, t->g.tiles, ntn, &tm, &t->tn);
    t->m0 = t->g.lo + (int)(tm << full.log);
  } else {
    index -= count;
    if (!group_of_tile(rest, index / ntn, &t->g)) return false;
    tile_of(index - t->g.before * ntn, t->g.tiles, ntn, &tm, &t->tn);
    const int rows = t->g.hi - t->g.lo;
    t->m0 = t->g.lo + (rows >> rest.log << rest.log) + (int)(tm << rest.rest_log);
  }
  return true;
}

TACO_DEV Epilogue of_group(const Epilogue& all, int g) {
  Epilogue e = all;
  if (e.bias.p) e.bias.p = static_cast<char*>(e.bias.p) + g * e.bias.ld * (e.bias.dt == kBF16 ? 2 : 4);
  return e;
}

// Forward products (w's k contiguous), and dx = dz w (BK_). Only as many
// workgroups as the groups have tiles do anything. Where tiles are few, K is
// cut into a.parts parts of a.part, whose sums go to a.partials
// [parts][a.rest tiles] for k_experts_join.
template <class TL, bool BK_, bool GATED, bool RAGGED, bool DIRECT>
TACO_DEV void experts_tile(const GemmArgs& a, const RowTile& r, int64_t b_rows, unsigned part, float* sums) {
  constexpr int BM = TL::BM, kCols = GATED ? TL::BN / 2 : TL::BN;
  const int64_t k0 = part * a.part;
  Tile t;
  t.m0 = r.m0;
  t.n0 = (int)r.tn * kCols;
  t.N = a.N;
  t.rows = r.g.hi - r.m0 < BM ? r.g.hi - r.m0 : BM;
  t.cols = a.N - t.n0 < kCols ? a.N - t.n0 : kCols;
  t.K = a.parts > 1 && a.K - k0 > a.part ? a.part : a.K - k0;
  t.a = a.a.p + r.m0 * a.a.ld + k0;
  t.b = a.b.p + r.g.g * b_rows * a.b.ld + (BK_ ? t.n0 + k0 * a.b.ld : t.n0 * a.b.ld + k0);
  t.b2 = GATED ? t.b + (int64_t)a.N * a.b.ld : t.b;
  t.lda = a.a.ld * (DIRECT ? 2 : 1);
  t.ldb = a.b.ld * (DIRECT ? 2 : 1);
  t.part = sums;
  sum_tile<TL, false, BK_, GATED, Bf16, RAGGED, DIRECT>(of_group(a.e, r.g.g), t);
}
template <class TL, bool BK_, bool GATED, bool DIRECT>
TACO_DEV void experts(const GemmArgs& a, const Groups& gr, int64_t b_rows, unsigned block) {
  using TR = typename RestOf<TL>::Type;
  static_assert(TL::kThreads == TR::kThreads && TL::BN == TR::BN && TR::kLdsBytes <= TL::kLdsBytes, "one launch");
  constexpr int kCols = GATED ? TL::BN / 2 : TL::BN;
  const unsigned ntn = (unsigned)(a.N + kCols - 1) / kCols;
  const GroupTiles<kFullTiles> full(gr, log2_of(TL::BM), log2_of(TR::BM));
  const GroupTiles<kRestTiles> rest(gr, log2_of(TL::BM), log2_of(TR::BM));
  // the full tiles' parts, then the others'
  const unsigned count = full.all() * ntn, more = rest.all() * ntn;
  unsigned tile, part = 0;
  if (block < count * a.parts) {
    tile = xcd_ordered(block, count * a.parts);
    if (a.parts > 1) part = tile / count, tile %= count;
  } else {
    block -= count * a.parts;
    if (block >= more * a.parts) return;
    tile = xcd_ordered(block, more * a.parts);
    if (a.parts > 1) part = tile / more, tile %= more;
    tile += count;
  }
  RowTile r;
  if (!locate(full, rest, ntn, tile, &r)) return;
  float* sums = nullptr;
  if (a.parts > 1) {
    if (tile >= a.rest) return;
    sums = a.partials + ((int64_t)part * a.rest + tile) * (TL::BM * TL::BN);
  }
  if (r.full) experts_tile<TL, BK_, GATED, false, DIRECT>(a, r, b_rows, part, sums);
  else experts_tile<TR, BK_, GATED, true, DIRECT>(a, r, b_rows, part, sums);
}
// DIRECT: x and w of any alignment.
template <class TL, bool BK_, bool GATED, bool DIRECT>
__global__ __launch_bounds__(TL::kThreads, 2) void k_experts(GemmArgs a, Groups gr, int64_t b_rows) {
  experts<TL, BK_, GATED, DIRECT>(a, gr, b_rows, blockIdx.x);
}

// Joins the parts of a tile's sums, in order, and finishes: a workgroup takes
// some rows of a tile, a lane eight columns.
template <class TL, bool GATED>
__global__ __launch_bounds__(256) void k_experts_join(GemmArgs a, Groups gr) {
  using TR = typename RestOf<TL>::Type;
  constexpr int BN = TL::BN, kCols = GATED ? BN / 2 : BN, kOcts = kCols / 8, kRows = 256 / kOcts;
  const unsigned ntn = (unsigned)(a.N + kCols - 1) / kCols;
  const GroupTiles<kFullTiles> full(gr, log2_of(TL::BM), log2_of(TR::BM));
  const GroupTiles<kRestTiles> rest(gr, log2_of(TL::BM), log2_of(TR::BM));
  RowTile r;
  if (!locate(full, rest, ntn, blockIdx.x, &r)) return;
  const int row = (int)blockIdx.y * kRows + (int)threadIdx.x / kOcts, col = (int)threadIdx.x % kOcts * 8;
  const int m = r.m0 + row, n = (int)r.tn * kCols + col;
  if (row >= (r.full ? TL::BM : TR::BM) || m >= r.g.hi || n >= a.N) return;
  float z[8], u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = 0.0f, u[i] = 0.0f;
  for (unsigned p = 0; p < a.parts; ++p) {
    const float* at = a.partials + (((int64_t)p * a.rest + blockIdx.x) * TL::BM + row) * BN + col;
    float f[8];
    load8(at, kF32, 0, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += f[i];
    if (GATED) {
      load8(at, kF32, kCols, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += f[i];
    }
  }
  const Epilogue e = of_group(a.e, r.g.g);
  if (GATED) finish_gated(e, a.N, m, n, a.N - n, z, u);
  else finish(e, m, n, a.N - n, z);
}

// The place-th largest group (the first of equals first), so that the longest
// sums begin first; the place-th group if there are more than a wave's lanes.
struct OneGroup {
  int g, lo, hi;
  TACO_DEV OneGroup(const Groups& gr, int place) {
    if (gr.count > kWave) {
      g = place;
      lo = offset_at(gr, g);
      hi = offset_at(gr, g + 1);
      return;
    }
    const int lane = (int)threadIdx.x % kWave;
    const int first = lane < gr.count ? offset_at(gr, lane) : 0, end = lane < gr.count ? offset_at(gr, lane + 1) : 0;
    const int rows = end - first;
    int before = 0;
    for (int i = 0; i < gr.count; ++i) {
      const int other = __builtin_amdgcn_readlane(rows, i);
      before += other > rows || (other == rows && i < lane);
    }
    g = __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < gr.count && before == place));
    lo = (int)lane_value((unsigned)first, g);
    hi = (int)lane_value((unsigned)end, g);
  }
};

// dw[g] = the product of dz and x over the group's rows; zeros if it has none.
// Whole tiles of 16-bit outputs are streamed past the caches (8 groups of 2 x 4096 x
// 4096, 8192 rows, all gradients 1092 us, kept in them 1120).
// A group's tiles take as long as it has rows, so each XCD has an eighth of
// every group's (a range of its own, where there are enough of them).
TACO_DEV unsigned dw_blocks(unsigned per) { return per < 2 * kXcds ? per : (per + kXcds - 1) / kXcds * kXcds; }
template <class TL, bool SINGLE = false>
TACO_DEV void experts_dw(const GemmArgs& a, const Groups& gr, unsigned block) {
  constexpr int BM = TL::BM, BN = TL::BN;
  const unsigned ntm = (unsigned)((a.M + BM - 1) / BM), ntn = (unsigned)((a.N + BN - 1) / BN);
  const unsigned per = ntm * ntn, blocks = dw_blocks(per), in_group = block % blocks;
  const unsigned index = blocks == per ? in_group : in_group % kXcds * (blocks / kXcds) + in_group / kXcds;
  if (index >= per) return;
  const OneGroup group(gr, (int)(block / blocks));
  const int g = group.g, lo = group.lo, hi = group.hi;
  unsigned tm, tn;
  tile_of(index, ntm, ntn, &tm, &tn);
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
  sum_tile<TL, true, true, false, Bf16, SINGLE, false, SINGLE>(e, t);
}
template <class TL>
__global__ __launch_bounds__(TL::kThreads, 2) void k_experts_dw(GemmArgs a, Groups gr) {
  experts_dw<TL>(a, gr, blockIdx.x);
}
// Sums of few rows: a tile's time is that of its loads, one after the other, and
// of its stores, so four workgroups share a CU.
__global__ __launch_bounds__(TilesSmall::kThreads, 4) void k_experts_dw_short(GemmArgs a, Groups gr) {
  experts_dw<TilesSmall, true>(a, gr, blockIdx.x);
}

// Few rows: of each group that has any, 16 * TM at a time. Workgroups that walk
// several column sets of a group with the next one's weights under way were
// slower (8 rows over 64 groups of 2 x 1024 x 2048 17.5 us, 16.3 so).
template <int TM, bool GATED, bool ANY>
__global__ __launch_bounds__(kFewWaves * kWave) void k_experts_few(GemmArgs a, Groups gr, int64_t b_rows) {
  const unsigned ntn = (unsigned)(a.N + a.cols - 1) / (unsigned)a.cols;
  const GroupTiles<kAllTiles> gt(gr, 31);   // one tile to a group
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
  const Epilogue e = of_group(a.e, g.g);
  for (int m = g.lo; m < g.hi; m += 16 * TM) {
    f.m0 = m;
    f.rows = g.hi - m < 16 * TM ? g.hi - m : 16 * TM;
    f.a = reinterpret_cast<const char*>(a.a.p + m * a.a.ld);
    few_rows_product<TM, GATED, Bf16, ANY>(e, f);
  }
}

// ------------------------------------------- backward of activations, dbias --

// dz, and the sums over ranges of 2^log rows of one group each (a gated layer has
// no bias: its dz comes from k_act_back).
__global__ __launch_bounds__(256) void k_experts_act_back(ActBackArgs a, Groups gr, int log, unsigned slabs, unsigned bound) {
  const GroupTiles<kAllTiles> gt(gr, log);
  const unsigned range = blockIdx.x / slabs;
  Group g;
  if (range >= bound || !group_of_tile(gt, range, &g)) return;
  const int64_t first = g.lo + ((int64_t)(range - g.before) << log), end = first + (int64_t(1) << log);
  act_back<false>(a, first, end < g.hi ? end : g.hi, range, blockIdx.x % slabs);
}

// Group g's sums of those, in order; zeros for a group without rows. `block`
// takes 64 columns; `sums`: kSumParts * kWave floats of LDS.
struct DbiasArgs {
  const float* partials;
  int N;
  Mat dbias;        // p null: not wanted
  unsigned bound;   // ranges that there is room for
  int log;          // of a range's rows
};
template <int WAVES>
TACO_DEV void experts_dbias(const DbiasArgs& a, const Groups& gr, unsigned block, int g, float* sums) {
  const GroupTiles<kAllTiles> gt(gr, a.log);
  // ranges before the lane that has the group, and before it in that lane
  const int lane = g / gt.per;
  unsigned before = lane_value(gt.upto - gt.mine, lane);
  for (int i = lane * gt.per; i < g; ++i) before += gt.tiles(offset_at(gr, i), offset_at(gr, i + 1));
  const unsigned tiles = gt.tiles(offset_at(gr, g), offset_at(gr, g + 1));
  ColumnSumArgs s;
  s.in = a.partials + (int64_t)before * a.N;
  s.ld = a.N;
  s.second = 0;
  s.count = before <= a.bound && tiles <= a.bound - before ? (int)tiles : 0;
  s.cols = a.N;
  s.out[0] = {static_cast<char*>(a.dbias.p) + g * a.dbias.ld * (a.dbias.dt == kBF16 ? 2 : 4), a.N, a.dbias.dt};
  column_sum<WAVES>(s, block, 0, sums);
}
__global__ __launch_bounds__(256) void k_experts_dbias(DbiasArgs a, Groups gr) {
  __shared__ float sums[kSumParts * kWave];
  experts_dbias<4>(a, gr, blockIdx.x, (int)blockIdx.y, sums);
}

// All gradients in one launch: dx's `count_dx` workgroups, dw's `count_dw`, and
// the biases'. dx's sums are the longer ones as a rule, so dw's tiles fill
// what dx leaves of the device at its end (8192 rows over 8 groups of 2 x 4096 x
// 4096 1073 to 1133 us with the activation's 64; as two launches 1126; large and small
// groups' tiles of dw in turn instead of the largest first 1273). FEW: few rows to a group, dw's sums
// are short (SINGLE) and dx takes the way with less LDS (DIRECT), so that three
// workgroups share a CU: 2000 rows over 32 groups of 520 x 1000 42.3 us with two,
// 35.4.
template <class TLX, class TLW, bool DIRECT, bool FEW>
__global__ __launch_bounds__(TLW::kThreads, FEW ? 3 : 2) void k_experts_back(GemmArgs dx, GemmArgs dw, DbiasArgs db, Groups gr,
                                                                   int64_t b_rows, unsigned count_dx, unsigned count_dw) {
  static_assert(TLX::kThreads == TLW::kThreads, "one launch");
  extern __shared__ __attribute__((aligned(1024))) uint16_t lds[];
  unsigned b = blockIdx.x;
  if (b < count_dx) {
    experts<TLX, true, false, DIRECT>(dx, gr, b_rows, b);
  } else if ((b -= count_dx) < count_dw) {
    experts_dw<TLW, FEW>(dw, gr, b);
  } else {
    b -= count_dw;
    const unsigned slabs = (unsigned)(db.N + kWave - 1) / kWave;
    experts_dbias<TLW::kThreads / kWave>(db, gr, b % slabs, (int)(b / slabs), reinterpret_cast<float*>(lds));
  }
}

// ----------------------------------------------------------------- launch --

// Tiles of 2^log rows that the groups can have at most.
static int64_t most_tiles(const Groups& g, int log) {
  const int64_t used = std::min(g.count, g.rows);   // groups with rows
  return (g.rows + used * ((int64_t(1) << log) - 1)) >> log;
}

// Whether a forward product takes the kernel for few rows, which reads a group's
// rows again for every 16 of its columns, or tiles. In us, that kernel and tiles:
// gated 2 x 1024 x 2048, 8 rows over 64 groups 16.0 and 17.7, 16 rows over 8 13.4
// and 16.0, 32 rows over 64 39.2 and 30.6; 4096 x 4096, 3 groups, 4 rows 10.0 and
// 13.6, 8 groups, 8 rows 36.0 and 31.8, 32 rows 57.5 and 41.2; 520 x 1000, 8 groups,
// 32 rows 8.6 and 12.3.
bool few_rows_experts(const Groups& g, int64_t n, int64_t k, bool gated) {
  return g.rows <= 4 || (g.rows <= kFewRows && g.rows * (gated ? 2 : 1) * n * k <= int64_t(1) << 26);
}

// Row tiles of k_experts at most: full ones, and those of the rows left.
template <class TL>
static int64_t most_row_tiles(const Groups& g) {
  using TR = typename RestOf<TL>::Type;
  const int64_t used = std::min(g.count, g.rows);
  if (TL::BM == TR::BM) return most_tiles(g, log2_of(TL::BM));
  return g.rows / TL::BM + std::min<int64_t>(TL::BM / TR::BM * used, most_tiles(g, log2_of(TR::BM)));
}
// A launch has fewer than 2^32 threads.
static bool fits_launch(int64_t workgroups, int threads) { return workgroups * threads < int64_t(1) << 32; }

// Which tiles the rows of groups take (dx, and forward products that are not of
// few rows). Large ones where they fill the device and most groups have a whole
// one or two: 8 groups of 2 x 4096 x 4096, 256 rows to a group 170 us, in small tiles
// 214 (350 rows 238 and 274; 175 rows 172 either way).
enum Shape { kFlat, kTall, kSmall, kLarge };
static Shape shape_of(const Groups& g, int64_t wide) {
  const int64_t rows = g.rows / g.count;
  if (rows <= 32) return kFlat;
  if (rows <= 64) return kTall;
  return rows >= 256 && g.rows * wide >= int64_t(192) << 16 ? kLarge : kSmall;
}

// The same for dx of N columns. A group of a few more rows than a tall tile's
// half leaves two low tiles beside its full ones, and of the largest sizes these
// would be more than a launch has threads (1024 groups of 33 rows, 1016800 columns:
// 5.2e9); small tiles are few enough at every size.
static Shape dx_shape(const Groups& g, int64_t N) {
  const Shape shape = shape_of(g, N);
  const int64_t ntn = (N + TilesTall::BN - 1) / TilesTall::BN;
  return shape == kTall && !fits_launch(most_row_tiles<TilesTall>(g) * ntn, TilesTall::kThreads) ? kSmall : shape;
}

// The same for a forward product of `ntn` columns of small tiles. More than one
// small tile to a CU: low tiles would read the weights of groups that have more
// rows than they hold in two rounds (8 groups of 2 x 2816 x 4096, 32, 48 and 64
// rows to a group 92, 99 and 94 us in flat or tall tiles, 78, 82 and 82 in small
// ones; but of 4096 x 4096, 256 small tiles, 48 and 64 rows 59 and 56, and 67 and 70).
static Shape forward_shape(const Groups& g, int64_t wide, int64_t ntn) {
  const Shape shape = shape_of(g, wide);
  if (shape == kLarge || g.rows / g.count < 32) return shape;
  return std::min(g.count, g.rows) * ntn > 256 ? kSmall : shape;
}

// Whether weights of another alignment are taken as they are, not copied: they
// are read about as often as the groups' rows fill tiles. 8 groups of 2 x 2816 x
// 4097, 256 rows to a group 252 us, copied 336; of 1000 x 1001, 512 rows 33.1 and
// 30.6. (Lines below 16 bytes are not taken.)
constexpr int kDirectRows = 512;
bool direct_experts(const Groups& g, int64_t wide) {
  return wide >= 8 && shape_of(g, wide) != kLarge && g.rows / g.count <= kDirectRows;
}

// Calls f(tiles) with the tiles of a shape.
template <class F>
static void with_tiles(Shape shape, F f) {
  switch (shape) {
    case kFlat: f(TilesFlat()); break;
    case kTall: f(TilesTall()); break;
    case kSmall: f(TilesSmall()); break;
    case kLarge: f(TilesLarge()); break;
  }
}

// How a product by group is cut; decided by the sizes alone, so that the
// workspace is known before the call.
struct ExpertsPlan {
  Shape shape;
  int64_t tiles;        // at most
  unsigned parts;       // of K
  int64_t part;
  size_t bytes;         // of partial sums
};
// `other`: us of the tiles of another product that run at the same time.
static ExpertsPlan plan_of(const Groups& g, Shape shape, int64_t N, int64_t K, bool gated, bool direct, double other) {
  ExpertsPlan p = {shape, 0, 1, K, 0};
  with_tiles(p.shape, [&](auto tiles) {
    using TL = decltype(tiles);
    const int64_t cols = gated ? TL::BN / 2 : TL::BN, ntn = (N + cols - 1) / cols, steps = (K + 63) / 64;
    p.tiles = most_row_tiles<TL>(g) * ntn;
    if (p.shape == kLarge) return;
    // about as many tiles as there will be: every group with rows has some left
    const double tiles_now = (double)((g.rows / TL::BM + std::min(g.count, g.rows)) * ntn);
    // two tiles to a CU, a step of either 0.6 us, by way of the registers 0.65 to 1.2; the parts' way
    // through memory at 4 TB/s, and a launch
    const double tile_us = 2.0 * TL::BM * TL::BN * sizeof(float) / 4e6, launch = 4.0;
    const double step = !direct ? 0.6 : TL::BM == TilesFlat::BM ? 0.65 : TL::BM == TilesTall::BM ? 0.9 : 1.2;
    double least = 0.0;
    for (int64_t parts = 1; parts <= std::max<int64_t>(1, std::min<int64_t>(steps / 4, 16)); ++parts) {
      const int64_t per = (steps + parts - 1) / parts;
      const double all = (tiles_now * (double)steps * step + other) / (2 * 256.0);
      const double t = std::max(all, (double)per * step) + (parts > 1 ? launch + tiles_now * (double)parts * tile_us : 0.0);
      if (parts == 1 || t < least) {
        least = t;
        p.parts = (unsigned)((steps + per - 1) / per);
        p.part = per * 64;
      }
    }
    if (p.parts > 1) p.bytes = (size_t)p.tiles * p.parts * TL::BM * TL::BN * sizeof(float);
  });
  return p;
}
static ExpertsPlan experts_plan(const Groups& g, int64_t N, int64_t K, bool gated, bool direct) {
  const int64_t wide = gated ? 2 * N : N;
  return plan_of(g, forward_shape(g, wide, (wide + TilesSmall::BN - 1) / TilesSmall::BN), N, K, gated, direct, 0.0);
}
// dx alone, and beside dw [wide, N] of every group, whose small tiles take about
// 5 us besides their steps.
static ExpertsPlan dx_plan(const Groups& g, int64_t N, int64_t wide, bool beside) {
  const double steps = (double)(g.rows / g.count) / 64.0;
  const double other = (double)(((wide + 127) / 128) * ((N + 127) / 128) * g.count) * (5.0 + 0.6 * steps);
  return plan_of(g, dx_shape(g, N), N, wide, false, false, beside ? other : 0.0);
}
static void set_experts_plan(GemmArgs* a, const ExpertsPlan& p, void* partials) {
  a->parts = p.parts;
  a->part = p.part;
  a->rest = (unsigned)p.tiles;
  a->partials = static_cast<float*>(partials);
}
size_t experts_partial_bytes(const Groups& g, int64_t N, int64_t K, bool gated, bool direct) {
  return g.rows == 0 ? 0 : experts_plan(g, N, K, gated, direct).bytes;
}

size_t experts_back_bytes(const Groups& g, int64_t N, int64_t wide) {
  return g.rows == 0 ? 0 : std::max(dx_plan(g, N, wide, false).bytes, dx_plan(g, N, wide, true).bytes);
}

template <class TL>
static void launch_experts_join(const GemmArgs& a, const Groups& g, hipStream_t s) {
  if constexpr (TL::BM < TilesLarge::BM) {   // (large tiles take all of K)
    if (a.parts <= 1) return;
    const int octs = (a.gated ? TL::BN / 2 : TL::BN) / 8, rows = 256 / octs;
    const dim3 grid(a.rest, (unsigned)((TL::BM + rows - 1) / rows));
    if (a.gated) hipLaunchKernelGGL((k_experts_join<TL, true>), grid, dim3(256), 0, s, a, g);
    else hipLaunchKernelGGL((k_experts_join<TL, false>), grid, dim3(256), 0, s, a, g);
  }
}

hipError_t launch_experts(const GemmArgs& args, const Groups& g, int64_t b_rows, void* partials, hipStream_t s) {
  if (g.rows == 0) return hipSuccess;
  GemmArgs a = args;
  if (!a.b.by_k && few_rows_experts(g, a.N, a.K, a.gated)) {
    a.cols = a.gated ? 8 : 16;
    const dim3 grid((unsigned)((a.N + a.cols - 1) / a.cols) * (unsigned)std::min(g.count, g.rows));
    const dim3 block(kFewWaves * kWave);
    auto few = [&](auto any) {
      constexpr bool ANY = any();
      if (a.gated) hipLaunchKernelGGL((k_experts_few<1, true, ANY>), grid, block, few_lds_bytes<1>(), s, a, g, b_rows);
      else hipLaunchKernelGGL((k_experts_few<1, false, ANY>), grid, block, few_lds_bytes<1>(), s, a, g, b_rows);
    };
    if (on_dwords(a.a.p, 2 * a.a.ld) && on_dwords(a.b.p, 2 * a.b.ld)) few(std::false_type());
    else few(std::true_type());
    return hipGetLastError();
  }
  const ExpertsPlan p = a.b.by_k ? dx_plan(g, a.N, a.K, false) : experts_plan(g, a.N, a.K, a.gated, a.direct);
  set_experts_plan(&a, p, partials);
  with_tiles(p.shape, [&](auto tiles) {
    using TL = decltype(tiles);
    auto launch = [&](auto direct) {
      const dim3 grid((unsigned)p.tiles * p.parts), block(TL::kThreads);
      constexpr size_t lds = direct() ? TL::kDirectLdsBytes : TL::kLdsBytes;
      if (a.b.by_k) hipLaunchKernelGGL((k_experts<TL, true, false, direct()>), grid, block, lds, s, a, g, b_rows);
      else if (a.gated) hipLaunchKernelGGL((k_experts<TL, false, true, direct()>), grid, block, lds, s, a, g, b_rows);
      else hipLaunchKernelGGL((k_experts<TL, false, false, direct()>), grid, block, lds, s, a, g, b_rows);
    };
    if constexpr (TL::BM < TilesLarge::BM) {
      if (a.direct) return launch(std::true_type()), launch_experts_join<TL>(a, g, s);
    }
    launch(std::false_type());
    launch_experts_join<TL>(a, g, s);
  });
  return hipGetLastError();
}

// Whether dw takes large tiles: there are enough of them, and the sums are long
// (8192 rows over 8 groups of 2 x 4096 x 4096 1092 us, 1299 in small ones; with 256
// rows to a group 497 either way, with 350 585 and 618).
static bool dw_large(const GemmArgs& a, const Groups& g) {
  return ((a.M + 255) / 256) * ((a.N + 255) / 256) * g.count >= 192 && g.rows / g.count >= 256;
}
template <class TL>
static unsigned dw_grid(const GemmArgs& a, const Groups& g) {
  const unsigned per = (unsigned)(((a.M + TL::BM - 1) / TL::BM) * ((a.N + TL::BN - 1) / TL::BN));
  return (per < 2 * kXcds ? per : (per + kXcds - 1) / kXcds * kXcds) * (unsigned)g.count;   // as dw_blocks()
}
// Whether dw takes the kernel for short sums, in a launch of its own: sums of
// about two steps at most, and many tiles (64 groups of 2048 x 2048: 512 rows in
// all 324 to 241 us, 8192 rows 447 to 369; but 32 of 512 x 1024, 1024 tiles, 33 to
// 40, and 8 of 3552 x 2248, 4032 tiles, 105 to 121: nothing runs beside it).
static bool dw_short(const GemmArgs& a, const Groups& g) {
  return g.rows / g.count <= 128 && ((a.M + 127) / 128) * ((a.N + 127) / 128) * g.count >= 8192;
}
template <class TL>
static void launch_dw_tiles(const GemmArgs& a, const Groups& g, hipStream_t s) {
  hipLaunchKernelGGL((k_experts_dw<TL>), dim3(dw_grid<TL>(a, g)), dim3(TL::kThreads), TL::kLdsBytes, s, a, g);
}
static void launch_dbias(const DbiasArgs& a, const Groups& g, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + kWave - 1) / kWave), (unsigned)g.count);
  hipLaunchKernelGGL(k_experts_dbias, grid, dim3(256), 0, s, a, g);
}

// Rows of a range: eight, as in a dense layer's pass, or more where there would
// be over 2048 ranges.
static int range_log(const Groups& g) {
  int log = 3;
  while (g.rows >> log > 2048) ++log;
  return log;
}
int64_t experts_back_ranges(const Groups& g) { return most_tiles(g, range_log(g)); }

hipError_t launch_experts_act_back(const ActBackArgs& a, const Groups& g, hipStream_t s) {
  const unsigned bound = (unsigned)experts_back_ranges(g), slabs = (unsigned)((a.N + 511) / 512);
  if (bound > 0) hipLaunchKernelGGL(k_experts_act_back, dim3(bound * slabs), dim3(256), 0, s, a, g, range_log(g), slabs, bound);
  return hipGetLastError();
}

hipError_t launch_experts_back(const GemmArgs* dx, const GemmArgs* dw, const float* sums, int64_t N, const Mat& dbias,
                               const Groups& g, int64_t b_rows, void* partials, hipStream_t s) {
  const DbiasArgs db = {sums, (int)N, dbias, (unsigned)experts_back_ranges(g), range_log(g)};
  const bool large_dw = dw && dw_large(*dw, g);
  const Shape shape = dx ? dx_shape(g, dx->N) : kFlat;
  const bool short_dw = dw && !large_dw && dw_short(*dw, g);
  const ExpertsPlan p = dx ? dx_plan(g, dx->N, dx->K, true) : ExpertsPlan();
  const unsigned count_dx = (unsigned)p.tiles * p.parts;
  const unsigned count_db = dbias.p ? (unsigned)((N + kWave - 1) / kWave) * (unsigned)g.count : 0;
  const unsigned count_dw = !dw ? 0 : large_dw ? dw_grid<TilesLarge>(*dw, g) : dw_grid<TilesSmall>(*dw, g);
  if (dx && dw && !short_dw && (shape == kLarge) == large_dw &&
      fits_launch((int64_t)count_dx + count_dw + count_db, large_dw ? TilesLarge::kThreads : TilesSmall::kThreads)) {
    GemmArgs x = *dx;
    set_experts_plan(&x, p, partials);
    with_tiles(shape, [&](auto tiles) {
      using TLX = decltype(tiles);
      using TLW = std::conditional_t<TLX::BM == TilesLarge::BM, TilesLarge, TilesSmall>;
      auto launch = [&](auto direct, auto few) {
        constexpr size_t lds = few() ? std::max(TLX::kDirectLdsBytes, TLW::kSingleLdsBytes) : TLW::kLdsBytes;
        hipLaunchKernelGGL((k_experts_back<TLX, TLW, direct(), few()>), dim3(count_dx + count_dw + count_db),
                           dim3(TLW::kThreads), lds, s, x, *dw, db, g, b_rows, count_dx, count_dw);
      };
      const std::true_type yes;
      const std::false_type no;
      if constexpr (TLX::BM < TilesSmall::BM) launch(yes, yes);
      else if constexpr (TLX::BM == TilesLarge::BM) launch(no, no);
      else if (x.direct) launch(yes, no);
      else launch(no, no);
      launch_experts_join<TLX>(x, g, s);
    });
    return hipGetLastError();
  }
  if (dbias.p) launch_dbias(db, g, s);
  if (dw) {
    if (large_dw) launch_dw_tiles<TilesLarge>(*dw, g, s);
    else if (short_dw)
      hipLaunchKernelGGL(k_experts_dw_short, dim3(dw_grid<TilesSmall>(*dw, g)), dim3(TilesSmall::kThreads),
                         TilesSmall::kSingleLdsBytes, s, *dw, g);
    else launch_dw_tiles<TilesSmall>(*dw, g, s);
  }
  return dx ? launch_experts(*dx, g, b_rows, partials, s) : hipGetLastError();
}

}  // namespace taco
