// Host-side interface between the layers' C ABI (layers_abi.hip) and their
// kernels. The ABI layer has validated what these structs carry.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace taco {

enum Dtype : int { kF32 = 0, kBF16 = 1 };

// A row-major matrix or a vector; p null: absent.
struct Mat {
  void* p;
  int64_t ld;   // elements from one row to the next
  int dt;
};

struct NormArgs {
  Mat x, weight, bias, y;
  int64_t rows;
  int cols;
  float eps;
  float *mean, *rstd;   // nullable
  int waves;            // that hold a row (set by launch_norm)
};

// Workgroups of the norm's kernels: two for each CU of the device. In the
// backward pass each adds up the weight's gradient over its rows and writes
// one partial sum per column, so their number is also what the workspace
// holds.
constexpr int kNormGroups = 512;

// out[0] [cols] = the sum of `count` rows of `in`, ld apart, and out[1] that of
// the columns `second` floats further on (zeros if count is 0; each may be
// absent).
struct ColumnSumArgs {
  const float* in;
  int64_t ld, second;
  int count, cols;
  Mat out[2];
};

struct NormBackArgs {
  Mat dy, x, weight, dx, dweight, dbias;
  int64_t rows;
  int cols;
  const float *mean, *rstd;
  float* partials;      // [groups][2][cols]
  int waves;            // that hold a row (set by launch_norm_back)
};

enum Act : int { kActNone = 0, kActGelu = 1, kActSilu = 2, kActRelu = 3 };

// What becomes of the sums z[m, n] of a matrix product.
struct Epilogue {
  Mat bias;       // [N], may be absent
  Mat residual;   // [M, N], may be absent
  Mat preact;     // receives z (+ bias), may be absent
  Mat out;
  int act;
};

// One operand of a matrix product, bf16: element (i, k) of its [rows, K] view
// is p[i * ld + k], or p[k * ld + i] if `by_k` (rows contiguous). Except for
// few rows, lines start on 16 bytes and may be read to the next multiple of
// eight elements, which hold zeros past the last k (k contiguous).
struct Operand {
  const uint16_t* p;
  int64_t ld;
  bool by_k;
};

// Up to two matrices to be copied with zeros up to the next multiple of eight
// elements.
struct PackArgs {
  struct One {
    Mat src;
    int64_t rows, cols;
    uint16_t* dst;
    int64_t ld;   // a multiple of 8
  } m[2];
  int count;
};
hipError_t launch_pack(const PackArgs& a, hipStream_t s);

// z[M, N] = a b^T over K, then the epilogue. With `gated`, N counts the output
// columns, b has 2 N rows (the gate's first) and the epilogue is
// out = act(z[:, :N]) * z[:, N:], preact [M, 2 N].
struct GemmArgs {
  Operand a, b;
  int64_t M;
  int N;
  int64_t K;
  bool gated;
  Epilogue e;
  // set by launch_gemm: the first `whole` tiles take all of K; K is cut into
  // `parts` parts of `part` (a multiple of 64) for the `rest` others, whose
  // sums go to partials [parts][rest] tiles in float32
  unsigned whole, rest, parts;
  int64_t part;
  float* partials;
  int cols;   // output columns of a workgroup, for few rows
};

// dz = dout * act'(z) (gated: both halves), and the column sums of dz.
struct ActBackArgs {
  Mat dout, z;          // [M, N], [M, N or 2 N]
  int64_t M;
  int N;
  int act;
  bool gated;
  uint16_t* dz;         // bf16 [M, ld_dz], null: not wanted
  int64_t ld_dz;
  float* partials;      // [act_back_groups][N], null: no column sums
};
int act_back_groups(int64_t M);

int norm_back_groups(int64_t rows, int64_t cols);
hipError_t launch_norm(NormArgs a, hipStream_t s);
hipError_t launch_norm_back(NormBackArgs a, hipStream_t s);
// Whether a forward product of this size takes the kernel for few rows, which
// takes operands as they are.
bool few_rows(int64_t M, int64_t N, int64_t K, bool gated);
// Bytes of partial sums that a product of this size takes (0: K is not cut).
size_t gemm_partial_bytes(int64_t M, int64_t N, int64_t K, bool gated);
hipError_t launch_gemm(GemmArgs a, void* partials, hipStream_t s);
// Both gradients of a projection, dx [M, K] and dw [wide, K], and a column
// sum, as one launch where they are small; gemm_pair_partial_bytes: for these,
// else 0.
size_t gemm_pair_partial_bytes(int64_t M, int64_t wide, int64_t K);
hipError_t launch_gemm_pair(GemmArgs dx, GemmArgs dw, const ColumnSumArgs& sum, void* partials, hipStream_t s);
hipError_t launch_act_back(const ActBackArgs& a, const PackArgs& p, hipStream_t s);   // and launch_pack's work
void launch_column_sum(const ColumnSumArgs& a, hipStream_t s);

}  // namespace taco
