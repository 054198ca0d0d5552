// Layer norm, forward and backward.
//
//   forward   y = (x - mean) rstd weight + bias
//   backward  dx = rstd (g - sum(g)/C - xhat sum(g xhat)/C),  g = dy weight,  xhat = (x - mean) rstd
//             dweight = sum over rows of dy xhat,  dbias = sum over rows of dy
//
// Memory bounds both: the forward pass reads and writes the tensor once, the
// backward pass reads two and writes one. A row therefore stays in registers,
// eight consecutive elements (one 16-byte load of bf16) per lane and step of
// its group of lanes, and the statistics are taken from there: first the mean,
// then the squares of the differences, which loses nothing where the mean is
// large against the spread. The row's last elements, fewer than eight, are
// held one per lane.
//
// Who holds a row: up to 512 elements, 16, 32 or 64 lanes of a wave, so that
// no lane is idle for long; wider, as many waves as one step takes (two steps
// above 8192 elements). A workgroup has up to sixteen waves, so it takes
// several narrow rows at a time, and walks the rows with a stride of the grid:
// weight and bias are read once, and the backward pass keeps its sums over
// rows in registers. What the bandwidth hangs on is the time from a row's
// loads to the next ones'. The forward pass has the next row's loads under way
// while a row is worked on; in the backward pass that measured slower (86
// against 62 us at 8192 x 5120), since the registers it takes cost a workgroup
// on every CU. Sums over lanes go by DPP and one LDS read per lane: with
// permutes through LDS the same passes took 47 and 78 us.
//
// Measured (bf16): forward 8192 x 5120 38 us (4.4 TB/s) with a part of three
// tensors in the Infinity Cache, 44 us (3.8 TB/s) without, 32768 x 5120 157 us
// (4.3 TB/s); backward with both sums 60 us (4.2 TB/s) and 201 us (5.0 TB/s).
// Forward 8192 x 5120 from float32 47 us (5.3 TB/s); 4096 x 16384 69 us (3.9).
// A copy of 1 GiB runs at 5.2 TB/s.
#include <type_traits>

#include "layers_device.h"
#include "layers_internal.h"

namespace taco {

constexpr int kNormThreads = 256;     // of the kernels that hold no whole rows
constexpr int kMaxNormWaves = 16;

// The lanes that share a row: L lanes of a wave, or (WIDE) `waves` whole ones.
template <int L, bool WIDE>
struct RowGroup {
  int lane;       // in the group
  int size;       // lanes of the group
  int in_block;   // groups before this one in the workgroup
  int blocks;     // groups of the workgroup
  TACO_DEV explicit RowGroup(int waves) {
    const int t = (int)threadIdx.x;
    size = WIDE ? waves * kWave : L;
    in_block = WIDE ? wave_in_group() / waves : t / L;
    lane = t - in_block * size;
    blocks = (int)blockDim.x / size;
  }
  // Sums of N values over the group. `slots`: [2][N * kMaxNormWaves] floats
  // of LDS, used in turn by successive calls (`turn`), so one barrier a call
  // is enough: a slot is written again only after the barrier of the call
  // between, which every wave passes after it has read it.
  template <int N>
  TACO_DEV void sum(float* v, float* slots, int turn) const {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<L>(v[i]);
    if constexpr (WIDE) {
      float* s = slots + (turn & 1) * N * kMaxNormWaves;
      if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i * kMaxNormWaves + wave_in_group()] = v[i];
      }
      lds_barrier();   // loads of the next row stay under way
      // lane l of each 16 takes wave l's sums
      const int waves = size / kWave, l = (int)threadIdx.x % 16;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = lanes_sum<16>(l < waves ? s[i * kMaxNormWaves + in_block * waves + l] : 0.0f);
    }
  }
};

// A lane's part of a row of `whole` eights and `rest` further elements.
template <int DT, int STEPS>
struct RowPart {
  Oct<DT> oct[STEPS];
  float last;
  TACO_DEV void load(const Mat& m, int64_t row, bool live, int lane, int size, int whole, int rest) {
    const int64_t at = row * m.ld;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      oct[i].clear();
      const int c = lane + i * size;
      if (live && c < whole) oct[i].load(m.p, at + c * 8);
    }
    last = live && lane < rest ? load1(m.p, DT, at + whole * 8 + lane) : 0.0f;
  }
  // Keeps the compiler from holding what one pass over the row has made of
  // these registers for the next pass: the row is kept as it was loaded.
  TACO_DEV void again() {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) oct[i].opaque();
  }
};

// Eight weights or biases; `absent` for each if there are none.
TACO_DEV void load8_or(const Mat& m, int c, float absent, float* f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = absent;
  if (m.p) load8(m.p, m.dt, c, f);
}

template <int DT, int L, bool WIDE, int STEPS>
__global__ __launch_bounds__(1024) void k_norm(NormArgs a) {
  __shared__ float slots[2 * kMaxNormWaves];
  const RowGroup<L, WIDE> g(a.waves);
  const int whole = a.cols / 8, rest = a.cols % 8;
  const float inv = 1.0f / (float)a.cols;
  float w[8], b[8];
  if (STEPS == 1 && g.lane < whole) {
    load8_or(a.weight, g.lane * 8, 1.0f, w);
    load8_or(a.bias, g.lane * 8, 0.0f, b);
  }
  const int64_t stride = (int64_t)gridDim.x * g.blocks;
  RowPart<DT, STEPS> x, next;
  next.load(a.x, (int64_t)blockIdx.x * g.blocks + g.in_block, (int64_t)blockIdx.x * g.blocks + g.in_block < a.rows,
            g.lane, g.size, whole, rest);
  for (int64_t first = (int64_t)blockIdx.x * g.blocks; first < a.rows; first += stride) {
    const int64_t row = first + g.in_block;
    const bool live = row < a.rows;
    x = next;
    next.load(a.x, row + stride, row + stride < a.rows, g.lane, g.size, whole, rest);
    float f[8], mean = x.last, var = 0.0f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      x.oct[i].get(f);   // zeros past the row's end
      mean += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    g.template sum<1>(&mean, slots, 0);
    mean *= inv;
    x.again();
    if (g.lane < rest) var = (x.last - mean) * (x.last - mean);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      x.oct[i].get(f);
      float v = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v = __builtin_fmaf(f[e] - mean, f[e] - mean, v);
      var += g.lane + i * g.size < whole ? v : 0.0f;
    }
    g.template sum<1>(&var, slots, 1);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(var, inv, a.eps));
    if (!live) continue;
    x.again();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int c = g.lane + i * g.size;
      if (c >= whole) continue;
      if (STEPS > 1) {
        load8_or(a.weight, c * 8, 1.0f, w);
        load8_or(a.bias, c * 8, 0.0f, b);
      }
      x.oct[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf((f[e] - mean) * rstd, w[e], b[e]);
      store8(a.y.p, a.y.dt, row * a.y.ld + c * 8, f);
    }
    if (g.lane < rest) {
      const int c = whole * 8 + g.lane;
      float t = (x.last - mean) * rstd;
      if (a.weight.p) t = t * load1(a.weight.p, a.weight.dt, c);
      if (a.bias.p) t = t + load1(a.bias.p, a.bias.dt, c);
      store1(a.y.p, a.y.dt, row * a.y.ld + c, t);
    }
    if (g.lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// dx, and with SUMS the sums over rows too: each lane keeps its part of
// dweight and dbias in registers until the end. Two steps per lane would not
// fit the registers with them: wider rows leave them to k_norm_back_sums.
template <int DT, int DY, int L, bool WIDE, int STEPS, bool SUMS>
__global__ __launch_bounds__(1024) void k_norm_back(NormBackArgs a) {
  static_assert(STEPS == 1 || !SUMS, "sums take one step per lane");
  __shared__ float slots[2 * 2 * kMaxNormWaves];
  extern __shared__ float sums[];   // [groups of rows][2][cols]
  const RowGroup<L, WIDE> g(a.waves);
  const int whole = a.cols / 8, rest = a.cols % 8;
  const float inv = 1.0f / (float)a.cols;
  // this lane's sums, and the weights they go with: eights and last element
  float w[8], dw[8], db[8], w_last = 1.0f, dw_last = 0.0f, db_last = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.0f, db[e] = 0.0f;
  if (STEPS == 1 && g.lane < whole) load8_or(a.weight, g.lane * 8, 1.0f, w);
  if (a.weight.p && g.lane < rest) w_last = load1(a.weight.p, a.weight.dt, whole * 8 + g.lane);
  struct {
    RowPart<DT, STEPS> x;
    RowPart<DY, STEPS> y;
    float mean, rstd;
  } now;
  auto load = [&](int64_t row, bool live) {
    now.x.load(a.x, row, live, g.lane, g.size, whole, rest);
    now.y.load(a.dy, row, live, g.lane, g.size, whole, rest);
    now.mean = live ? a.mean[row] : 0.0f;
    now.rstd = live ? a.rstd[row] : 0.0f;
  };
  const int64_t stride = (int64_t)gridDim.x * g.blocks;
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * g.blocks; first < a.rows; first += stride) {
    const int64_t row = first + g.in_block;
    const bool live = row < a.rows;
    load(row, live);
    float x[8], y[8], s[2] = {0.0f, 0.0f};
    // one element: sums of dy xhat, dy, g and g xhat
    auto add = [&](float x, float y, float w, float& dw, float& db, bool in) {
      x = in ? (x - now.mean) * now.rstd : 0.0f;
      if constexpr (SUMS) {
        dw = __builtin_fmaf(y, x, dw);
        db += y;
      }
      y *= w;
      s[0] += y;
      s[1] = __builtin_fmaf(y, x, s[1]);
    };
    if (rest > 0) add(now.x.last, now.y.last, w_last, dw_last, db_last, g.lane < rest && live);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int c = g.lane + i * g.size;
      now.x.oct[i].get(x);
      now.y.oct[i].get(y);
      if (c >= whole) continue;
      if (STEPS > 1) load8_or(a.weight, c * 8, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) add(x[e], y[e], w[e], dw[e], db[e], live);
    }
    if (a.dx.p == nullptr) continue;
    g.template sum<2>(s, slots, turn++);
    if (!live) continue;
    s[0] *= inv;
    s[1] *= inv;
    auto slope = [&](float x, float y, float w) {
      return (__builtin_fmaf(y, w, -s[0]) - (x - now.mean) * now.rstd * s[1]) * now.rstd;
    };
    now.x.again();
    now.y.again();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int c = g.lane + i * g.size;
      if (c >= whole) continue;
      now.x.oct[i].get(x);
      now.y.oct[i].get(y);
      if (STEPS > 1) load8_or(a.weight, c * 8, 1.0f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = slope(x[e], y[e], w[e]);
      store8(a.dx.p, a.dx.dt, row * a.dx.ld + c * 8, y);
    }
    if (g.lane < rest)
      store1(a.dx.p, a.dx.dt, row * a.dx.ld + whole * 8 + g.lane, slope(now.x.last, now.y.last, w_last));
  }
  if constexpr (SUMS) {
    // a workgroup's groups are added up in LDS, in order
    float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
    float* mine = g.blocks == 1 ? part : sums + g.in_block * 2 * a.cols;
    if (g.lane < whole) {
      keep8(mine + g.lane * 8, dw);
      keep8(mine + a.cols + g.lane * 8, db);
    }
    if (g.lane < rest) {
      mine[whole * 8 + g.lane] = dw_last;
      mine[a.cols + whole * 8 + g.lane] = db_last;
    }
    if (g.blocks == 1) return;
    __syncthreads();
    for (int i = (int)threadIdx.x; i < 2 * a.cols; i += (int)blockDim.x) {
      float t = 0.0f;
      for (int k = 0; k < g.blocks; ++k) t += sums[k * 2 * a.cols + i];
      part[i] = t;
    }
  }
}

// The sums over rows alone: a workgroup takes 2048 columns (blockIdx.y) of
// every gridDim.x-th row. Rows wider than 8192 thus read dy and x twice: 4096 x
// 16384 backward 162 us in both kernels (671 MB, 4.1 TB/s).
template <int DT, int DY>
__global__ __launch_bounds__(kNormThreads) void k_norm_back_sums(NormBackArgs a) {
  const int c = ((int)blockIdx.y * kNormThreads + (int)threadIdx.x) * 8, n = a.cols - c;
  if (n <= 0) return;
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.0f, db[e] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    Oct<DT> rx;
    Oct<DY> ry;
    rx.load(a.x.p, row * a.x.ld + c, n);
    ry.load(a.dy.p, row * a.dy.ld + c, n);
    const float mean = a.mean[row], rstd = a.rstd[row];
    float x[8], y[8];
    rx.get(x);
    ry.get(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[e] += y[e] * ((x[e] - mean) * rstd);
      db[e] += y[e];
    }
  }
  float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
  store8<false>(part, kF32, c, n, dw);
  store8<false>(part, kF32, a.cols + c, n, db);
}

// 512 rows of 2 x 5120 floats: 4.6 us, most of it the launch and two chains of
// loads.
__global__ __launch_bounds__(kSumParts * kWave) void k_column_sum(ColumnSumArgs a) {
  __shared__ float sums[kSumParts * kWave];
  column_sum<kSumParts>(a, blockIdx.x, blockIdx.y, sums);
}

void launch_column_sum(const ColumnSumArgs& a, hipStream_t s) {
  if (a.out[0].p == nullptr && a.out[1].p == nullptr) return;
  const dim3 grid((unsigned)((a.cols + kWave - 1) / kWave), a.out[1].p ? 2 : 1);
  hipLaunchKernelGGL(k_column_sum, grid, dim3(kSumParts * kWave), 0, s, a);
}

// How rows of `cols` elements are held.
struct NormShape {
  int lanes;     // of a wave that hold a row, or 64
  int waves;     // that hold a row (lanes == 64)
  int steps;
  int threads;   // of a workgroup
  int rows;      // that a workgroup takes at a time
};
static NormShape norm_shape(int cols) {
  NormShape n = {cols <= 128 ? 16 : cols <= 256 ? 32 : 64, 1, cols <= 8192 ? 1 : 2, kMaxNormWaves * kWave, 0};
  const int per = 8 * kWave * n.steps;
  n.waves = (cols + per - 1) / per;
  n.rows = n.lanes < kWave ? n.threads / n.lanes : kMaxNormWaves / n.waves;
  if (n.lanes == kWave) n.threads = n.rows * n.waves * kWave;
  return n;
}

// f(L, WIDE, STEPS as constants)
template <class F>
static void for_shape(const NormShape& n, F f) {
  using std::integral_constant;
  using std::true_type;
  using std::false_type;
  const integral_constant<int, 64> wave;
  const integral_constant<int, 1> one;
  if (n.lanes == 16) f(integral_constant<int, 16>(), false_type(), one);
  else if (n.lanes == 32) f(integral_constant<int, 32>(), false_type(), one);
  else if (n.waves == 1) f(wave, false_type(), one);
  else if (n.steps == 1) f(wave, true_type(), one);
  else f(wave, true_type(), integral_constant<int, 2>());
}

// Two workgroups on every CU take all rows.
static int64_t norm_groups(int64_t rows, const NormShape& n) {
  const int64_t blocks = (rows + n.rows - 1) / n.rows;
  return blocks < kNormGroups ? blocks : kNormGroups;
}

hipError_t launch_norm(NormArgs a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const NormShape n = norm_shape(a.cols);
  a.waves = n.waves;
  const dim3 grid((unsigned)norm_groups(a.rows, n)), block((unsigned)n.threads);
  for_shape(n, [&](auto l, auto wide, auto steps) {
    constexpr int L = l(), STEPS = steps();
    constexpr bool WIDE = wide();
    if (a.x.dt == kBF16) hipLaunchKernelGGL((k_norm<kBF16, L, WIDE, STEPS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_norm<kF32, L, WIDE, STEPS>), grid, block, 0, s, a);
  });
  return hipGetLastError();
}

int norm_back_groups(int64_t rows, int64_t cols) { return (int)norm_groups(rows, norm_shape((int)cols)); }

// f(the two element types as constants)
template <class F>
static void for_types(int x, int dy, F f) {
  using std::integral_constant;
  const integral_constant<int, kBF16> bf16;
  const integral_constant<int, kF32> f32;
  if (x == kBF16) dy == kBF16 ? f(bf16, bf16) : f(bf16, f32);
  else dy == kBF16 ? f(f32, bf16) : f(f32, f32);
}

hipError_t launch_norm_back(NormBackArgs a, hipStream_t s) {
  const NormShape n = norm_shape(a.cols);
  const int groups = (int)norm_groups(a.rows, n);
  const bool sums = a.dweight.p || a.dbias.p;
  a.waves = n.waves;
  if (groups > 0) {
    const dim3 grid((unsigned)groups), block((unsigned)n.threads);
    for_types(a.x.dt, a.dy.dt, [&](auto x, auto dy) {
      constexpr int X = x(), DY = dy();
      for_shape(n, [&](auto l, auto wide, auto steps) {
        constexpr int L = l(), STEPS = steps();
        constexpr bool WIDE = wide();
        if constexpr (STEPS == 1) {
          if (sums) {
            const size_t lds = n.rows > 1 ? (size_t)n.rows * 2 * (size_t)a.cols * sizeof(float) : 0;
            hipLaunchKernelGGL((k_norm_back<X, DY, L, WIDE, 1, true>), grid, block, lds, s, a);
            return;
          }
        } else if (sums) {
          constexpr int kCols = kNormThreads * 8;
          const dim3 slabs((unsigned)groups, (unsigned)((a.cols + kCols - 1) / kCols));
          hipLaunchKernelGGL((k_norm_back_sums<X, DY>), slabs, dim3(kNormThreads), 0, s, a);
          if (a.dx.p == nullptr) return;
        }
        hipLaunchKernelGGL((k_norm_back<X, DY, L, WIDE, STEPS, false>), grid, block, 0, s, a);
      });
    });
  }
  if (sums)
    launch_column_sum(ColumnSumArgs{a.partials, 2 * (int64_t)a.cols, a.cols, groups, a.cols, {a.dweight, a.dbias}}, s);
  return hipGetLastError();
}

}  // namespace taco
