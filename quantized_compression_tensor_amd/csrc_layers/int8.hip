// Projections in 8-bit integers: rows to codes, and the forward products of
// codes with a scale for each row of x (a token) and of w (an output channel),
//   z[m, n] = (sum over k of qx[m, k] qw[n, k]) sx[m] sw[n] + bias
// with the epilogues of linear.hip. The sums are whole numbers, exact in 32
// bits up to K = 131071 (2^31 / 2^14), so neither their order nor a cut of K
// changes a bit; a sum becomes a float with one rounding, and each scale is one
// more.
//
// The matrix cores take twice as many codes as bf16 elements at a time, in the
// same 16 bytes of a lane, so a product of codes is one of 16-bit elements with
// half the K to everything but the matrix instruction and the epilogue: tiles,
// stages of LDS, waits and plans are those of linear.hip.
// Measured in streams of calls: 8192^3 with bias and residual 431 to 456 us (2500
// TOP/s; the library's product of codes, without an epilogue, 515), bound by the
// matrix cores at the clock that power leaves (profiled 449 us, busy 0.67 of the
// time at 1.89 GHz); gated 4096 x 5120 x 5120 190 to 198 (2.2 PTOP/s, busy 0.64 at 2.1
// GHz). One row, 4096 x 4096: 8.0 us, 6.6 of them on the device; 24 rows, gated 2 x
// 1728 x 5120: 8.7. Large tiles that stay on their CU and load the next one's first
// steps during an epilogue were slower (8192^3 457 to 477 us).
#define TACO_DEVICE_CODE_ONLY
#include "linear.hip"

namespace taco {

// --------------------------------------------------------------- products --

// DIRECT: x and w of any alignment.
template <class TL, bool GATED, bool DIRECT>
__global__ __launch_bounds__(TL::kThreads, 2) void k_int8(GemmArgs a) {
  gemm<TL, false, false, GATED, Int8, DIRECT>(a, blockIdx.x);
}

template <class TL, bool GATED, bool DIRECT>
static void launch_tiles_int8(const GemmArgs& a, hipStream_t s) {
  constexpr size_t lds = DIRECT ? TL::kDirectLdsBytes : TL::kLdsBytes;
  hipLaunchKernelGGL((k_int8<TL, GATED, DIRECT>), dim3(a.whole + a.rest * a.parts), dim3(TL::kThreads), lds, s, a);
  if (a.rest == 0) return;
  const int octs = (GATED ? TL::BN / 2 : TL::BN) / 8, rows = 256 / octs;
  hipLaunchKernelGGL((k_join<TL, GATED, Int8>), dim3(a.rest, (unsigned)(TL::BM / rows)), dim3(256), 0, s, a);
}

// Products whose operands are not aligned take them from where they lie
// (DIRECT), in tiles of 32 or 64 rows, or copies of them in the other tiles,
// whichever a model of their times says is least. In us: a step of the direct
// tiles, in rounds of 256; parts of K, as in linear.hip's plan; a copy at 4 TB/s
// and its launch. (A CU holds four of the tiles of 32 rows, 40 KB of LDS and 110
// registers each, and three of 64, so more than 256 take less than their rounds
// say: of those, copies are taken a little early.) Tiles of 32 and of 64 rows, 3 bytes off: 200 rows by 4096
// x 4096 20.6 and 27.2, 301 by 1001 x 1285 12.1 and 14.7; but 100 by 4096 x 4096 21.9
// and 17.9 (copied 22.1). 8000 by 129 x 777 15.1, copied 19.4; 1000 by 6000 x 511
// 26.5 and 20.4.
struct Int8Plan {
  int height;               // of a tile
  unsigned tiles, parts;    // parts of K
  int64_t part;             // pairs of codes
  double us;
};
static Int8Plan int8_plan(int64_t M, int64_t N, int64_t K, bool gated) {
  Int8Plan p = {0, 0, 1, 0, 0.0};
  const int64_t cols = gated ? 64 : 128, steps = (K + 127) / 128;
  for (const int height : {TilesFlat::BM, TilesTall::BM}) {
    const int64_t tiles = (M + height - 1) / height * ((N + cols - 1) / cols);
    const double step = height == TilesFlat::BM ? 0.65 : 0.85, part_us = 2.0 * height * 128 * sizeof(float) / 4e6;
    for (int64_t parts = 1; parts <= std::max<int64_t>(1, std::min<int64_t>(steps / 4, 16)); ++parts) {
      const int64_t per = (steps + parts - 1) / parts;
      const double rounds = (double)((tiles * parts + 255) / 256);
      const double us = rounds * (double)per * step + (parts > 1 ? 5.0 + (double)(tiles * parts) * part_us : 0.0);
      if (p.height == 0 || us < p.us) p = {height, (unsigned)tiles, (unsigned)((steps + per - 1) / per), per * 64, us};
    }
  }
  return p;
}
bool direct_int8(int64_t M, int64_t N, int64_t K, bool gated) {
  const Int8Plan p = int8_plan(M, N, K, gated);
  const double copy = 3.5 + 2.0 * (double)((M + (gated ? 2 * N : N)) * K) / 4e6;
  // (a launch has fewer than 2^32 threads)
  return (int64_t)p.tiles * p.parts < int64_t(1) << 20 && p.us < copy + gemm_plan_us(M, N, (K + 1) / 2, gated);
}
size_t direct_int8_bytes(int64_t M, int64_t N, int64_t K, bool gated) {
  const Int8Plan p = int8_plan(M, N, K, gated);
  return p.parts == 1 ? 0 : (size_t)p.tiles * p.parts * (size_t)p.height * 128 * sizeof(float);
}

// As few_rows(), for rows of half the bytes: 48 rows by 4096 x 4096 11.8 us, in
// tiles 13.8; 64 by 8192 x 1024 8.5 and 11.2; but 64 by 1248 x 6912 17.2 and 13.8.
bool few_rows_int8(int64_t M, int64_t N, int64_t K, bool gated) {
  const int64_t weights = (gated ? 2 : 1) * N * K;
  return M <= 4 || (M <= 64 && weights * M <= int64_t(1) << 30);
}

hipError_t launch_gemm_int8(Int8Kernel kernel, GemmArgs a, void* partials, hipStream_t s) {
  if (kernel == kInt8Few) {
    const dim3 grid(set_few_columns(&a)), block(kFewWaves * kWave);
    auto few = [&](auto tiles, auto any) {
      constexpr int TM = tiles();
      constexpr bool ANY = any();
      if (a.gated) hipLaunchKernelGGL((k_few_rows<TM, true, Int8, ANY>), grid, block, few_lds_bytes<TM>(), s, a);
      else hipLaunchKernelGGL((k_few_rows<TM, false, Int8, ANY>), grid, block, few_lds_bytes<TM>(), s, a);
    };
    auto with = [&](auto any) {
      if (a.M <= 16) few(std::integral_constant<int, 1>(), any);
      else if (a.M <= 32) few(std::integral_constant<int, 2>(), any);
      else few(std::integral_constant<int, 4>(), any);
    };
    if (on_dwords(a.a.p, a.a.ld) && on_dwords(a.b.p, a.b.ld)) with(std::false_type());
    else with(std::true_type());
    return hipGetLastError();
  }
  auto launch = [&](auto tiles, auto direct) {
    using TL = decltype(tiles);
    if (a.gated) launch_tiles_int8<TL, true, direct()>(a, s);
    else launch_tiles_int8<TL, false, direct()>(a, s);
  };
  if (kernel == kInt8Direct) {
    const Int8Plan p = int8_plan(a.M, a.N, a.K, a.gated);
    a.whole = p.parts == 1 ? p.tiles : 0;
    a.rest = p.tiles - a.whole;
    a.parts = p.parts;
    a.part = p.part;
    a.partials = static_cast<float*>(partials);
    if (p.height == TilesFlat::BM) launch(TilesFlat(), std::true_type());
    else launch(TilesTall(), std::true_type());
  } else if (set_gemm_plan(&a, partials)) {
    launch(TilesLarge(), std::false_type());
  } else {
    launch(TilesSmall(), std::false_type());
  }
  return hipGetLastError();
}

// ----------------------------------------------------------------- packing --

// Copies matrices of bytes so that rows start on 16 bytes and hold a multiple
// of 16, zeros past the last; a lane takes 16. Rows may start anywhere.
__global__ __launch_bounds__(256) void k_pack_int8(PackArgs a) {
  const PackArgs::One m = a.m[blockIdx.y];
  const int64_t parts = (m.cols + 15) / 16, total = m.rows * parts;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = total <= UINT32_MAX ? (uint32_t)i / (uint32_t)parts : i / parts;
    const int64_t c = (i - row * parts) * 16, left = m.cols - c;
    const u32x4 v = load_part<Int8>(static_cast<const char*>(m.src.p) + row * m.src.ld + c, left < 16 ? (int)left : 16);
    *reinterpret_cast<u32x4*>(reinterpret_cast<char*>(m.dst) + row * m.ld + c) = v;
  }
}

hipError_t launch_pack_int8(const PackArgs& a, hipStream_t s) {
  int64_t most = 0;
  for (int i = 0; i < a.count; ++i) most = std::max(most, a.m[i].rows * ((a.m[i].cols + 15) / 16));
  const unsigned blocks = (unsigned)std::min<int64_t>((most + 255) / 256, 4096);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_pack_int8, dim3(blocks, (unsigned)a.count), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ------------------------------------------------------------ rows to codes --

// The largest magnitude of a row, as the bits of its absolute value: these are
// in the order of the values, with infinity and then NaN above all others.
TACO_DEV unsigned magnitude(float f) { return __builtin_bit_cast(unsigned, f) & 0x7FFFFFFFu; }

template <int LANES>
TACO_DEV unsigned lanes_max(unsigned v) {
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) {
    const unsigned o = (unsigned)__shfl_xor((int)v, d, kWave);
    v = o > v ? o : v;
  }
  return v;
}

// A row's scale A / 127 and what its elements are multiplied by, (1 / A) 127 in
// two roundings, as a program that has the reciprocals makes it (the codec
// INT8_SYM has 127 / A in one: codes next to a half may be one apart). The scale is
// at most 2^-24 of its value off, the multiplier 2^-23 up to A = 2^126 and 2^-21.6
// above, where 1 / A is subnormal (2^-22, and one rounding). Rows below kTiny are
// zeros; rows with an infinity or NaN have that as their scale, and codes of zero.
struct RowScale {
  float scale, inv;
  TACO_DEV explicit RowScale(unsigned bits) {
    const float largest = __builtin_bit_cast(float, bits);
    const bool finite = bits < 0x7F800000u, zero = finite && largest < kTiny;
    scale = zero ? 0.0f : finite ? largest / 127.0f : largest;
    inv = finite && !zero ? 1.0f / largest * 127.0f : 0.0f;
  }
  // |x inv| is at most 127 (1 + 2^-21), below 127.5, so the codes need no clamp
  TACO_DEV int code(float x) const { return inv == 0.0f ? 0 : rne_int(x * inv); }
};
TACO_DEV unsigned four_codes(const float* f, const RowScale& s) {
  return (unsigned)(s.code(f[0]) & 255) | (unsigned)(s.code(f[1]) & 255) << 8 | (unsigned)(s.code(f[2]) & 255) << 16 |
         (unsigned)s.code(f[3]) << 24;
}

constexpr int kQuantizeSteps = 4;   // eights of a row that a lane holds

// A row is held by `waves` waves, four eights to a lane at most; where it is
// longer (SECOND) its parts are read again for the codes. Bound by memory: 8192 x
// 8192 bf16 32.0 us on the device (6.3 TB/s), 38.6 in a stream of calls over three
// inputs, which the caches do not hold (5.2 TB/s, a copy's rate). Narrow rows are
// held by LANES lanes of a wave, or most of it would have nothing to do (64767 x
// 205 bf16 51.0 us with a wave to a row, 11.7; 30000 x 500 25.0 and 11.7).
template <int DT, bool SECOND, int LANES>
__global__ __launch_bounds__(1024) void k_quantize(QuantizeArgs a, int waves) {
  __shared__ unsigned largest[2][16];   // used in turn, so that one barrier a row is enough
  static_assert(LANES == kWave || !SECOND, "a narrow row is read once");
  const int wave = wave_in_group(), size = LANES < kWave ? LANES : waves * kWave, first_wave = wave / waves * waves;
  const int lane = LANES < kWave ? (int)threadIdx.x % LANES : (int)threadIdx.x - first_wave * kWave;
  const int rows_at_once = (int)blockDim.x / size;
  int turn = 0;
  for (int64_t block = (int64_t)blockIdx.x * rows_at_once; block < a.rows; block += (int64_t)gridDim.x * rows_at_once) {
    const int64_t row = block + (LANES < kWave ? (int)threadIdx.x / LANES : wave / waves);
    const bool live = row < a.rows;
    const char* x = static_cast<const char*>(a.x.p) + (live ? row : 0) * a.x.ld * (DT == kBF16 ? 2 : 4);
    char* q = static_cast<char*>(a.q.p) + (live ? row : 0) * a.q.ld;
    const int64_t octs = live ? (a.cols + 7) / 8 : 0, per = (int64_t)kQuantizeSteps * size;
    Oct<DT> o[kQuantizeSteps];
    auto load = [&](int64_t from) {
#pragma unroll
      for (int i = 0; i < kQuantizeSteps; ++i) {
        const int64_t c = from + lane + i * size, left = a.cols - 8 * c;
        o[i].clear();
        if (c < octs) o[i].load(x, 8 * c, left < 8 ? (int)left : 8);
      }
    };
    unsigned m = 0;
    auto look = [&] {
#pragma unroll
      for (int i = 0; i < kQuantizeSteps; ++i) {
        float f[8];
        o[i].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const unsigned b = magnitude(f[e]);
          m = b > m ? b : m;
        }
      }
    };
    load(0);
    look();
    if constexpr (SECOND) {
      for (int64_t from = per; from < octs; from += per) {
        load(from);
        look();
      }
    }
    m = lanes_max<LANES>(m);
    if (LANES == kWave && waves > 1) {
      if (lane % kWave == 0) largest[turn][wave] = m;
      __syncthreads();
      for (int w = 0; w < waves; ++w) m = largest[turn][first_wave + w] > m ? largest[turn][first_wave + w] : m;
      turn ^= 1;
    }
    const RowScale s(m);
    auto store = [&](int64_t from) {
#pragma unroll
      for (int i = 0; i < kQuantizeSteps; ++i) {
        const int64_t c = from + lane + i * size, left = a.cols - 8 * c;
        if (c >= octs) continue;
        float f[8];
        o[i].get(f);
        const unsigned w[2] = {four_codes(f, s), four_codes(f + 4, s)};
        if (left >= 8) {
          __builtin_memcpy(q + 8 * c, w, 8);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < left) q[8 * c + e] = (char)(w[e / 4] >> (8 * (e % 4)));
        }
      }
    };
    if constexpr (SECOND) {
      for (int64_t from = 0; from < octs; from += per) {
        load(from);
        store(from);
      }
    } else {
      store(0);
    }
    if (live && lane == 0) a.scale[row] = s.scale;
  }
}

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s) {
  const int64_t octs = (a.cols + 7) / 8;
  int waves = 1;
  while (waves < 16 && (int64_t)waves * kWave * kQuantizeSteps < octs) waves *= 2;
  const bool second = (int64_t)waves * kWave * kQuantizeSteps < octs;
  const int lanes = octs <= 8 * kQuantizeSteps ? 8 : octs <= 16 * kQuantizeSteps ? 16 : waves * kWave;
  const int per = std::max(1, 256 / lanes);
  const dim3 grid((unsigned)std::min<int64_t>((a.rows + per - 1) / per, 1 << 16)), block((unsigned)(per * lanes));
  auto launch = [&](auto dt) {
    constexpr int DT = dt();
    if (lanes == 8) hipLaunchKernelGGL((k_quantize<DT, false, 8>), grid, block, 0, s, a, waves);
    else if (lanes == 16) hipLaunchKernelGGL((k_quantize<DT, false, 16>), grid, block, 0, s, a, waves);
    else if (second) hipLaunchKernelGGL((k_quantize<DT, true, kWave>), grid, block, 0, s, a, waves);
    else hipLaunchKernelGGL((k_quantize<DT, false, kWave>), grid, block, 0, s, a, waves);
  };
  if (a.x.dt == kBF16) launch(std::integral_constant<int, kBF16>());
  else launch(std::integral_constant<int, kF32>());
  return hipGetLastError();
}

}  // namespace taco
