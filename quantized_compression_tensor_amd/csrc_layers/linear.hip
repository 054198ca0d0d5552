// Matrix products of a linear layer, forward and backward, with their
// epilogues: z[M, N] = sum over k of a[m, k] b[n, k], and then
//   linear   out = act(z + bias) + residual
//   gated    out = act(z[:, :F]) * z[:, F:]
// in float32 on the bf16 matrix cores. An operand lies in memory with its k
// contiguous (x and W of the forward pass) or with its rows contiguous (W for
// dx = dz W, dz and x for dw = dz^T x).
#include "layers_device.h"
#include "layers_internal.h"

namespace taco {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define TACO_LDS __attribute__((address_space(3)))

// ------------------------------------------------------------ activations --

TACO_DEV float act_value(float t, int act) {
  switch (act) {
    case kActGelu: return 0.5f * t * (1.0f + erff(t * 0.70710678118654752f));
    case kActSilu: return t / (1.0f + expf(-t));
    case kActRelu: return t < 0.0f ? 0.0f : t;   // NaN stays
    default: return t;
  }
}

// act'(t): Phi(t) + t phi(t); s (1 + t (1 - s)) with s = 1 / (1 + exp(-t)); t > 0.
TACO_DEV float act_slope(float t, int act) {
  switch (act) {
    case kActGelu:
      return 0.5f * (1.0f + erff(t * 0.70710678118654752f)) + t * (expf(-0.5f * t * t) * 0.39894228040143268f);
    case kActSilu: {
      const float s = 1.0f / (1.0f + expf(-t));
      return s * (1.0f + t * (1.0f - s));
    }
    case kActRelu: return t > 0.0f ? 1.0f : 0.0f;
    default: return 1.0f;
  }
}

// --------------------------------------------------------------- epilogue --

// Eight neighbouring columns n ... of row m, of which `count` exist.
TACO_DEV void finish(const Epilogue& e, int64_t m, int n, int count, float* z) {
  if (e.bias.p) {
    float b[8];
    load8(e.bias.p, e.bias.dt, n, count, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
  }
  if (e.preact.p) store8(e.preact.p, e.preact.dt, m * e.preact.ld + n, count, z);
  if (e.act != kActNone) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], e.act);
  }
  if (e.residual.p) {
    float r[8];
    load8(e.residual.p, e.residual.dt, m * e.residual.ld + n, count, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
  }
  store8(e.out.p, e.out.dt, m * e.out.ld + n, count, z);
}
// The same of a gated layer with `width` output columns: z gate, u the other.
TACO_DEV void finish_gated(const Epilogue& e, int width, int64_t m, int n, int count, float* z, float* u) {
  if (e.preact.p) {
    store8(e.preact.p, e.preact.dt, m * e.preact.ld + n, count, z);
    store8(e.preact.p, e.preact.dt, m * e.preact.ld + width + n, count, u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = act_value(z[i], e.act) * u[i];
  store8(e.out.p, e.out.dt, m * e.out.ld + n, count, z);
}

// ------------------------------------------------------------------ tiles --

template <int BM_, int BN_, int WGM_, int WGN_>
struct Tiles {
  static constexpr int BM = BM_, BN = BN_, BK = 64, WGM = WGM_, WGN = WGN_;
  static constexpr int kThreads = kWave * WGM * WGN;
  static constexpr int TM = BM / WGM / 32, TN = BN / WGN / 32;   // 32 x 32 MFMA tiles of a wave
  static constexpr int kStage = (BM + BN) * BK;                  // elements of one LDS stage
};
using TilesLarge = Tiles<256, 256, 2, 4>;
using TilesSmall = Tiles<128, 128, 2, 2>;

// A tile of R rows by 64 k in LDS, without padding, in chunks of 8 elements.
// A matrix product reads a chunk column (k contiguous) or a block of 4 k by 16
// rows (rows contiguous, transposed by the LDS read itself); the chunks of a
// line are permuted by an xor of their number so that either read touches all
// LDS banks evenly.
//   k contiguous      line = row, 8 chunks of 8 k;  chunk c at c ^ ((row >> 1) & 7):
//                     16 neighbouring rows of one chunk column fill 256 bytes
//   rows contiguous   line = k, R / 8 chunks of 8 rows;  chunk c at
//                     c ^ (4 (k & 3) + 2 ((k >> 3) & 1)): the 4 k of a read,
//                     64 bytes each, fill 256 bytes
template <bool BY_K, int R>
struct LdsTile {
  static constexpr int kPerLine = BY_K ? R / 8 : 8;
  static constexpr int kChunks = R * 8;
  static TACO_DEV int swizzle(int line) {
    return BY_K ? 4 * (line & 3) + 2 * ((line >> 3) & 1) : (line >> 1) & 7;
  }
  // Line and chunk of the chunk at position q of the tile in LDS.
  static TACO_DEV int line_of(int q) { return q / kPerLine; }
  static TACO_DEV int chunk_of(int q) { return (q % kPerLine) ^ swizzle(q / kPerLine); }
  // Operand of a 32 x 32 x 16 product: lane l holds row r0 + l % 32 and the
  // eight k of 16 kk + 8 (l / 32).
  static TACO_DEV bf16x8 operand(const uint16_t* t, int r0, int kk, int lane) {
    if constexpr (!BY_K) {
      const int r = r0 + (lane & 31), c = 2 * kk + (lane >> 5);
      return *reinterpret_cast<const bf16x8*>(t + r * 64 + (c ^ swizzle(r)) * 8);
    } else {
      // a read takes, for each 16 lanes, 4 k of 16 rows from addresses of 4
      // rows each, and gives lane i of them the four k of row i
      const int k = 16 * kk + 8 * (lane >> 5) + ((lane >> 2) & 3);
      const int r = r0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
      union {
        s16x4 h[2];
        bf16x8 v;
      } u;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int kl = k + 4 * i;
        const uint16_t* at = t + kl * R + ((r >> 3) ^ swizzle(kl)) * 8 + (r & 7);
        u.h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TACO_LDS s16x4*)at);
      }
      return u.v;
    }
  }
};

// Moves one tile's chunks of one operand from memory into LDS.
template <bool BY_K, int R, int NT>
struct Loader {
  using Tile = LdsTile<BY_K, R>;
  static constexpr int kPer = Tile::kChunks / NT;
  static_assert(Tile::kChunks % NT == 0, "whole chunks for every thread");
  u32x4 reg[kPer];
  TACO_DEV void load(const uint16_t* p, int64_t ld, int rows, int64_t k0, int64_t K, int tid) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = tid + i * NT, line = Tile::line_of(q), c = Tile::chunk_of(q);
      const int64_t k = k0 + (BY_K ? line : 8 * c);
      const int r = BY_K ? 8 * c : line;
      const int64_t left = BY_K ? (k < K ? rows - r : 0) : (r < rows ? K - k : 0);
      Oct<kBF16> o;
      o.load(p, BY_K ? k * ld + r : r * ld + k, left > 8 ? 8 : (int)left);
      reg[i] = o.v;
    }
  }
  TACO_DEV void store(uint16_t* t, int tid) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<u32x4*>(t + (tid + i * NT) * 8) = reg[i];
  }
};

template <class TL, bool AK, bool BK_>
__global__ __launch_bounds__(TL::kThreads) void k_gemm(GemmArgs a) {
  constexpr int BM = TL::BM, BN = TL::BN, BK = TL::BK, TM = TL::TM, TN = TL::TN, NT = TL::kThreads;
  extern __shared__ __attribute__((aligned(1024))) uint16_t lds[];
  const int tid = (int)threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
  const int wm = wave / TL::WGN, wn = wave % TL::WGN;
  const int ntn = (a.N + BN - 1) / BN;
  const int64_t m0 = (int64_t)(blockIdx.x / ntn) * BM;
  const int n0 = (int)(blockIdx.x % ntn) * BN;
  const int rows_a = (int)(a.M - m0 < BM ? a.M - m0 : BM), rows_b = a.N - n0 < BN ? a.N - n0 : BN;
  const uint16_t* pa = a.a.p + (AK ? m0 : m0 * a.a.ld);
  const uint16_t* pb = a.b.p + (BK_ ? n0 : n0 * a.b.ld);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  Loader<AK, BM, NT> la;
  Loader<BK_, BN, NT> lb;
  la.load(pa, a.a.ld, rows_a, 0, a.K, tid);
  lb.load(pb, a.b.ld, rows_b, 0, a.K, tid);
  for (int64_t k0 = 0; k0 < a.K; k0 += BK) {
    __syncthreads();
    la.store(lds, tid);
    lb.store(lds + BM * BK, tid);
    __syncthreads();
    if (k0 + BK < a.K) {
      la.load(pa, a.a.ld, rows_a, k0 + BK, a.K, tid);
      lb.load(pb, a.b.ld, rows_b, k0 + BK, a.K, tid);
    }
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      bf16x8 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = LdsTile<AK, BM>::operand(lds, wm * TM * 32 + i * 32, kk, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = LdsTile<BK_, BN>::operand(lds + BM * BK, wn * TN * 32 + j * 32, kk, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();
  // Accumulator e of lane l holds row 8 (e / 4) + 4 (l / 32) + e % 4, column
  // l % 32 of its tile. Each wave turns 32 rows at a time round through its
  // own part of LDS, so that a lane has eight neighbouring columns of a row.
  constexpr int kCols = TN * 32, kLd = kCols + 4;
  float* turn = reinterpret_cast<float*>(lds) + wave * 32 * kLd;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        turn[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * kLd + j * 32 + (lane & 31)] = acc[i][j][e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    constexpr int kLanes = kCols / 8;   // per row
    for (int r = lane / kLanes; r < 32; r += kWave / kLanes) {
      const int c = (lane % kLanes) * 8, n = n0 + wn * kCols + c;
      const int64_t m = m0 + (wm * TM + i) * 32 + r;
      float z[8];
      *reinterpret_cast<f32x4*>(z) = *reinterpret_cast<const f32x4*>(turn + r * kLd + c);
      *reinterpret_cast<f32x4*>(z + 4) = *reinterpret_cast<const f32x4*>(turn + r * kLd + c + 4);
      if (m < a.M && n < a.N) finish(a.e, m, n, a.N - n, z);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// The gated layer: a tile of 64 output columns, the gate's 64 rows of b and
// then the other projection's.
__global__ __launch_bounds__(256) void k_gated(GemmArgs a) {
  constexpr int BM = 128, BN = 128, BK = 64, NT = 256, F = BN / 2;
  extern __shared__ __attribute__((aligned(1024))) uint16_t lds[];
  const int tid = (int)threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
  const int wm = wave / 2, wn = wave % 2;
  const int ntn = (a.N + F - 1) / F;
  const int64_t m0 = (int64_t)(blockIdx.x / ntn) * BM;
  const int n0 = (int)(blockIdx.x % ntn) * F;
  const int rows_a = (int)(a.M - m0 < BM ? a.M - m0 : BM), rows_b = a.N - n0 < F ? a.N - n0 : F;
  const uint16_t* pa = a.a.p + m0 * a.a.ld;
  const uint16_t* pg = a.b.p + n0 * a.b.ld;
  const uint16_t* pu = a.b.p + (n0 + (int64_t)a.N) * a.b.ld;
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  Loader<false, BM, NT> la;
  Loader<false, F, NT> lg, lu;
  for (int64_t k0 = 0; k0 < a.K; k0 += BK) {
    la.load(pa, a.a.ld, rows_a, k0, a.K, tid);
    lg.load(pg, a.b.ld, rows_b, k0, a.K, tid);
    lu.load(pu, a.b.ld, rows_b, k0, a.K, tid);
    __syncthreads();
    la.store(lds, tid);
    lg.store(lds + BM * BK, tid);
    lu.store(lds + (BM + F) * BK, tid);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BK / 16; ++kk) {
      bf16x8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = LdsTile<false, BM>::operand(lds, wm * 64 + i * 32, kk, lane);
        fb[i] = LdsTile<false, F>::operand(lds + (BM + i * F) * BK, wn * 32, kk, lane);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();
  constexpr int kLd = 64 + 4;
  float* turn = reinterpret_cast<float*>(lds) + wave * 32 * kLd;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        turn[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * kLd + j * 32 + (lane & 31)] = acc[i][j][e];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int r = lane / 4; r < 32; r += 16) {
      const int c = (lane % 4) * 8, n = n0 + wn * 32 + c;
      const int64_t m = m0 + (wm * 2 + i) * 32 + r;
      float z[8], u[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<f32x4*>(z + 4 * h) = *reinterpret_cast<const f32x4*>(turn + r * kLd + c + 4 * h);
        *reinterpret_cast<f32x4*>(u + 4 * h) = *reinterpret_cast<const f32x4*>(turn + r * kLd + 32 + c + 4 * h);
      }
      if (m < a.M && n < a.N) finish_gated(a.e, a.N, m, n, a.N - n, z, u);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

template <class TL>
static void launch_tiles(const GemmArgs& a, hipStream_t s) {
  const int64_t tiles = ((a.M + TL::BM - 1) / TL::BM) * (((int64_t)a.N + TL::BN - 1) / TL::BN);
  const dim3 grid((unsigned)tiles), block(TL::kThreads);
  const size_t stage = TL::kStage * 2, turn = (size_t)TL::kThreads / kWave * 32 * (TL::TN * 32 + 4) * 4;
  const size_t lds = stage > turn ? stage : turn;
  if (!a.a.by_k && !a.b.by_k) hipLaunchKernelGGL((k_gemm<TL, false, false>), grid, block, lds, s, a);
  else if (!a.a.by_k) hipLaunchKernelGGL((k_gemm<TL, false, true>), grid, block, lds, s, a);
  else hipLaunchKernelGGL((k_gemm<TL, true, true>), grid, block, lds, s, a);
}

hipError_t launch_gemm(const GemmArgs& a, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  if (a.gated) {
    const int64_t tiles = ((a.M + 127) / 128) * (((int64_t)a.N + 63) / 64);
    hipLaunchKernelGGL(k_gated, dim3((unsigned)tiles), dim3(256), 4 * 32 * 68 * 4, s, a);
  } else {
    launch_tiles<TilesSmall>(a, s);
  }
  return hipGetLastError();
}

// ------------------------------------------------- backward of activations --

// A workgroup takes 512 columns (blockIdx.y) of a range of rows, a wave every
// fourth row of them, a lane eight neighbouring columns. 64 rows are a range;
// more where there would be over kActMaxGroups ranges.
constexpr int kActRows = 64, kActMaxGroups = 1024;
int act_back_groups(int64_t M) {
  const int64_t g = (M + kActRows - 1) / kActRows;
  return (int)(g < kActMaxGroups ? g : kActMaxGroups);
}

template <bool GATED>
__global__ __launch_bounds__(256) void k_act_back(ActBackArgs a) {
  __shared__ float sums[4][512];
  const int lane = (int)threadIdx.x % kWave, wave = wave_in_group();
  const int c = ((int)blockIdx.y * kWave + lane) * 8, n = a.N - c;
  const int64_t per = (a.M + gridDim.x - 1) / gridDim.x, first = blockIdx.x * per;
  const int64_t end = first + per < a.M ? first + per : a.M;
  float db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) db[e] = 0.0f;
  for (int64_t m = first + wave; m < end; m += 4) {
    if (n <= 0) break;
    float d[8], z[8];
    load8(a.dout.p, a.dout.dt, m * a.dout.ld + c, n, d);
    if (GATED || a.act != kActNone) load8(a.z.p, a.z.dt, m * a.z.ld + c, n, z);
    if constexpr (GATED) {
      float u[8], dg[8];
      load8(a.z.p, a.z.dt, m * a.z.ld + a.N + c, n, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[e] = d[e] * u[e] * act_slope(z[e], a.act);
        d[e] = d[e] * act_value(z[e], a.act);
      }
      store8(a.dz, kBF16, m * a.ld_dz + c, n, dg);
      store8(a.dz, kBF16, m * a.ld_dz + a.N + c, n, d);
    } else {
      if (a.act != kActNone) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = d[e] * act_slope(z[e], a.act);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) db[e] += d[e];
      if (a.dz) store8(a.dz, kBF16, m * a.ld_dz + c, n, d);
    }
  }
  if (GATED || a.partials == nullptr) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[wave][lane * 8 + e] = db[e];
  __syncthreads();
  for (int i = (int)threadIdx.x; i < 512; i += 256) {
    const int col = (int)blockIdx.y * 512 + i;
    if (col < a.N)
      a.partials[(int64_t)blockIdx.x * a.N + col] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
  }
}

hipError_t launch_act_back(const ActBackArgs& a, hipStream_t s) {
  const int groups = act_back_groups(a.M);
  if (groups > 0) {
    const dim3 grid((unsigned)groups, (unsigned)((a.N + 511) / 512));
    if (a.gated) hipLaunchKernelGGL((k_act_back<true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_act_back<false>), grid, dim3(256), 0, s, a);
  }
  launch_column_sum(a.partials, a.N, groups, a.N, a.dbias, s);
  return hipGetLastError();
}

}  // namespace taco
