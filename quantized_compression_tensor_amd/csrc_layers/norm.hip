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
// large against the spread.
//
// Rows of up to 512 elements take 16, 32 or 64 lanes of one wave, so that
// their sums need no barrier and no lane is idle for long; wider rows take a
// workgroup, with one step up to 8192 elements and two beyond.
#include "layers_device.h"
#include "layers_internal.h"

namespace taco {

constexpr int kNormThreads = 256;     // workgroups whose waves hold whole rows
constexpr int kMaxNormWaves = 16;
constexpr int64_t kNormMaxGroups = 1 << 20;   // of the forward pass: a launch has less than 2^32 threads

// Which of a row's elements this thread holds, and how its group adds up.
// L: lanes per row inside a wave; WIDE: the row takes the whole workgroup.
template <int L, bool WIDE>
struct RowGroup {
  int lane;       // in the group
  int size;       // lanes of the group
  int in_block;   // groups before this one in the workgroup
  int blocks;     // groups of the workgroup
  TACO_DEV RowGroup() {
    const int t = (int)threadIdx.x;
    if constexpr (WIDE) {
      lane = t;
      size = (int)blockDim.x;
      in_block = 0;
      blocks = 1;
    } else {
      lane = t % L;
      size = L;
      in_block = t / L;
      blocks = (int)blockDim.x / L;
    }
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
      const int wave = wave_in_group(), waves = (int)blockDim.x / kWave;
      if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i * kMaxNormWaves + wave] = v[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float t = 0.0f;
        for (int w = 0; w < waves; ++w) t += s[i * kMaxNormWaves + w];
        v[i] = t;
      }
    }
  }
};

template <int DT, int L, bool WIDE, int STEPS>
__global__ __launch_bounds__(WIDE ? 1024 : kNormThreads) void k_norm(NormArgs a) {
  __shared__ float slots[2 * kMaxNormWaves];
  const RowGroup<L, WIDE> g;
  for (int64_t first = (int64_t)blockIdx.x * g.blocks; first < a.rows; first += (int64_t)gridDim.x * g.blocks) {
  const int64_t row = first + g.in_block;
  const bool live = row < a.rows;   // with WIDE, always
  const int64_t r = live ? row : 0;
  Oct<DT> raw[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int c = (g.lane + i * g.size) * 8;
    raw[i].load(a.x.p, r * a.x.ld + c, a.cols - c);
  }
  const float inv = 1.0f / (float)a.cols;
  float f[STEPS][8];
  float mean = 0.0f;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    raw[i].get(f[i]);   // elements past the row's end are zeros
#pragma unroll
    for (int e = 0; e < 8; ++e) mean += f[i][e];
  }
  g.template sum<1>(&mean, slots, 0);
  mean *= inv;
  float var = 0.0f;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int n = a.cols - (g.lane + i * g.size) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[i][e] = f[i][e] - mean;
      var += e < n ? f[i][e] * f[i][e] : 0.0f;
    }
  }
  g.template sum<1>(&var, slots, 1);
  const float rstd = 1.0f / __builtin_sqrtf(var * inv + a.eps);
  if (!live) return;   // only in the last round
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int c = (g.lane + i * g.size) * 8, n = a.cols - c;
    if (n <= 0) break;
    float w[8], b[8];
    if (a.weight.p) load8(a.weight.p, a.weight.dt, c, n, w);
    if (a.bias.p) load8(a.bias.p, a.bias.dt, c, n, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float t = f[i][e] * rstd;
      if (a.weight.p) t = t * w[e];
      if (a.bias.p) t = t + b[e];
      f[i][e] = t;
    }
    store8(a.y.p, a.y.dt, r * a.y.ld + c, n, f[i]);
  }
  if (g.lane == 0) {
    if (a.mean) a.mean[r] = mean;
    if (a.rstd) a.rstd[r] = rstd;
  }
  }
}

// dx, and with SUMS the sums over rows too: each workgroup takes every
// gridDim-th group of rows and keeps its part of dweight and dbias in
// registers until the end. With one step per lane everything a row needs fits
// the registers; wider rows leave the sums to k_norm_back_sums.
template <int DT, int DY, int L, bool WIDE, int STEPS, bool SUMS>
__global__ __launch_bounds__(WIDE ? 1024 : kNormThreads) void k_norm_back(NormBackArgs a) {
  static_assert(STEPS == 1 || !SUMS, "sums take one step per lane");
  __shared__ float slots[2 * 2 * kMaxNormWaves];
  const RowGroup<L, WIDE> g;
  const float inv = 1.0f / (float)a.cols;
  float w[8], dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.0f, dw[e] = 0.0f, db[e] = 0.0f;
  if (STEPS == 1 && a.weight.p) load8(a.weight.p, a.weight.dt, g.lane * 8, a.cols - g.lane * 8, w);
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * g.blocks; first < a.rows; first += (int64_t)gridDim.x * g.blocks) {
    const int64_t row = first + g.in_block;
    const bool live = row < a.rows;   // with WIDE, always
    Oct<DT> rx[STEPS];
    Oct<DY> ry[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int c = (g.lane + i * g.size) * 8, n = live ? a.cols - c : 0;
      rx[i].load(a.x.p, row * a.x.ld + c, n);
      ry[i].load(a.dy.p, row * a.dy.ld + c, n);
    }
    const float mean = live ? a.mean[row] : 0.0f, rstd = live ? a.rstd[row] : 0.0f;
    float x[STEPS][8], y[STEPS][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int c = (g.lane + i * g.size) * 8, n = live ? a.cols - c : 0;
      rx[i].get(x[i]);
      ry[i].get(y[i]);
      if (STEPS > 1 && a.weight.p) load8(a.weight.p, a.weight.dt, c, a.cols - c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[i][e] = e < n ? (x[i][e] - mean) * rstd : 0.0f;
        if constexpr (SUMS) {
          dw[e] += y[i][e] * x[i][e];
          db[e] += y[i][e];
        }
        y[i][e] = y[i][e] * w[e];
        s[0] += y[i][e];
        s[1] += y[i][e] * x[i][e];
      }
    }
    if (a.dx.p) {
      g.template sum<2>(s, slots, turn++);
      s[0] *= inv;
      s[1] *= inv;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int c = (g.lane + i * g.size) * 8, n = live ? a.cols - c : 0;
        if (n <= 0) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] = (y[i][e] - s[0] - x[i][e] * s[1]) * rstd;
        store8(a.dx.p, a.dx.dt, row * a.dx.ld + c, n, y[i]);
      }
    }
  }
  if constexpr (SUMS) {
    float* part = a.partials + (int64_t)blockIdx.x * 2 * a.cols;
    if constexpr (WIDE) {
      const int c = g.lane * 8, n = a.cols - c;
      if (n <= 0) return;
      store8(part, kF32, c, n, dw);
      store8(part + a.cols, kF32, c, n, db);
    } else {
      // the workgroup's groups are added up in LDS, in order
      constexpr int kGroups = kNormThreads / L;
      __shared__ float sums[kGroups][2][L * 8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sums[g.in_block][0][g.lane * 8 + e] = dw[e];
        sums[g.in_block][1][g.lane * 8 + e] = db[e];
      }
      __syncthreads();
      for (int i = (int)threadIdx.x; i < 2 * a.cols; i += kNormThreads) {
        const int v = i >= a.cols, c = i - v * a.cols;
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) t += sums[k][v][c];
        part[i] = t;
      }
    }
  }
}

// The sums over rows alone: a workgroup takes 2048 columns (blockIdx.y) of
// every gridDim.x-th row.
template <int DT, int DY>
__global__ __launch_bounds__(kNormThreads) void k_norm_back_sums(NormBackArgs a) {
  const int c = ((int)blockIdx.y * kNormThreads + (int)threadIdx.x) * 8, n = a.cols - c;
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.0f, db[e] = 0.0f;
  if (n <= 0) return;
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
  store8(part, kF32, c, n, dw);
  store8(part + a.cols, kF32, c, n, db);
}

// Sums of `count` rows of `cols` floats, `ld` apart: 64 columns per workgroup,
// its four waves every fourth row each.
struct ColumnSumArgs {
  const float* in;
  int64_t ld;
  int count, cols;
  Mat out;
};
__global__ __launch_bounds__(kNormThreads) void k_column_sum(ColumnSumArgs a) {
  __shared__ float sums[4][kWave];
  const int lane = (int)threadIdx.x % kWave, wave = wave_in_group();
  const int c = (int)blockIdx.x * kWave + lane;
  float t = 0.0f;
  if (c < a.cols)
    for (int r = wave; r < a.count; r += 4) t += a.in[r * a.ld + c];
  sums[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && c < a.cols)
    store1(a.out.p, a.out.dt, c, (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]));
}

void launch_column_sum(const float* in, int64_t ld, int count, int64_t cols, const Mat& out, hipStream_t s) {
  if (out.p == nullptr) return;
  const ColumnSumArgs a = {in, ld, count, (int)cols, out};
  hipLaunchKernelGGL(k_column_sum, dim3((unsigned)((cols + kWave - 1) / kWave)), dim3(kNormThreads), 0, s, a);
}

// Threads of a workgroup that holds one row: one step of eight elements each
// where 1024 are enough.
static int wide_steps(int cols) { return cols <= 8192 ? 1 : 2; }
static int wide_threads(int cols) {
  const int per = 8 * wide_steps(cols);
  return ((cols + per - 1) / per + kWave - 1) / kWave * kWave;
}
// Lanes per row inside a wave; 0: the row takes a workgroup.
static int narrow_lanes(int cols) { return cols <= 128 ? 16 : cols <= 256 ? 32 : cols <= 512 ? 64 : 0; }

// f(L, WIDE, STEPS as constants)
template <class F>
static void for_shape(int cols, F f) {
  using std::integral_constant;
  switch (narrow_lanes(cols)) {
    case 16: return f(integral_constant<int, 16>(), std::false_type(), integral_constant<int, 1>());
    case 32: return f(integral_constant<int, 32>(), std::false_type(), integral_constant<int, 1>());
    case 64: return f(integral_constant<int, 64>(), std::false_type(), integral_constant<int, 1>());
    default: break;
  }
  if (wide_steps(cols) == 1) f(integral_constant<int, 64>(), std::true_type(), integral_constant<int, 1>());
  else f(integral_constant<int, 64>(), std::true_type(), integral_constant<int, 2>());
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  for_shape(a.cols, [&](auto l, auto wide, auto steps) {
    constexpr int L = l(), STEPS = steps();
    constexpr bool WIDE = wide();
    const int per_block = WIDE ? 1 : kNormThreads / L;
    const int64_t blocks = (a.rows + per_block - 1) / per_block;
    const dim3 grid((unsigned)(blocks < kNormMaxGroups ? blocks : kNormMaxGroups));
    const dim3 block(WIDE ? wide_threads(a.cols) : kNormThreads);
    if (a.x.dt == kBF16) hipLaunchKernelGGL((k_norm<kBF16, L, WIDE, STEPS>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_norm<kF32, L, WIDE, STEPS>), grid, block, 0, s, a);
  });
  return hipGetLastError();
}

int norm_back_groups(int64_t rows, int64_t cols) {
  const int lanes = narrow_lanes((int)cols);
  const int64_t per_block = lanes ? kNormThreads / lanes : 1;
  const int64_t blocks = (rows + per_block - 1) / per_block;
  return (int)(blocks < kNormBackGroups ? blocks : kNormBackGroups);
}

// f(the two element types as constants)
template <class F>
static void for_types(int x, int dy, F f) {
  using std::integral_constant;
  const integral_constant<int, kBF16> bf16;
  const integral_constant<int, kF32> f32;
  if (x == kBF16) dy == kBF16 ? f(bf16, bf16) : f(bf16, f32);
  else dy == kBF16 ? f(f32, bf16) : f(f32, f32);
}

hipError_t launch_norm_back(const NormBackArgs& a, hipStream_t s) {
  const int groups = norm_back_groups(a.rows, a.cols);
  const bool sums = a.dweight.p || a.dbias.p;
  if (groups > 0) {
    for_types(a.x.dt, a.dy.dt, [&](auto x, auto dy) {
      constexpr int X = x(), DY = dy();
      for_shape(a.cols, [&](auto l, auto wide, auto steps) {
        constexpr int L = l(), STEPS = steps();
        constexpr bool WIDE = wide();
        const dim3 grid((unsigned)groups), block(WIDE ? wide_threads(a.cols) : kNormThreads);
        if constexpr (STEPS == 1) {
          if (sums) {
            hipLaunchKernelGGL((k_norm_back<X, DY, L, WIDE, 1, true>), grid, block, 0, s, a);
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
  if (!sums) return hipGetLastError();
  const int64_t ld = 2 * (int64_t)a.cols;
  launch_column_sum(a.partials, ld, groups, a.cols, a.dweight, s);
  launch_column_sum(groups ? a.partials + a.cols : nullptr, ld, groups, a.cols, a.dbias, s);
  return hipGetLastError();
}

}  // namespace taco
