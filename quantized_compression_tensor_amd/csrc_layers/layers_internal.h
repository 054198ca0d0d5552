// Host-side interface between the layers' C ABI (layers_abi.hip) and their
// kernels. The ABI layer has validated what these structs carry.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace taco {

enum Dtype : int { kF32 = 0, kBF16 = 1, kI8 = 2 };

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
  const float *row_scale, *col_scale;   // [M], [weight rows]: for products of 8-bit codes
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
  // set by a product's launch (launch_gemm, launch_gemm_pair, launch_gemm_int8,
  // launch_experts, launch_experts_back): the first `whole` tiles take all of K;
  // K is cut into `parts` parts of `part` (a multiple of 64) for the `rest`
  // others, whose sums go to partials [parts][rest] tiles in float32
  unsigned whole, rest, parts;
  int64_t part;
  float* partials;
  int cols;   // output columns of a workgroup, for few rows
  bool direct;   // a and b may start and end anywhere (products by group only)
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
// The time of a product that its plan goes by, without its launch and epilogue.
double gemm_plan_us(int64_t M, int64_t N, int64_t K, bool gated);
// Fills in the plan of a product; whether its tiles are the large ones.
bool set_gemm_plan(GemmArgs* a, void* partials);
// Fills in the columns of a workgroup of the kernel for few rows; its grid.
unsigned set_few_columns(GemmArgs* a);
// Both gradients of a projection, dx [M, K] and dw [wide, K], and a column
// sum, as one launch where they are small; gemm_pair_partial_bytes: for these,
// else 0.
size_t gemm_pair_partial_bytes(int64_t M, int64_t wide, int64_t K);
hipError_t launch_gemm_pair(GemmArgs dx, GemmArgs dw, const ColumnSumArgs& sum, void* partials, hipStream_t s);
hipError_t launch_act_back(const ActBackArgs& a, const PackArgs& p, hipStream_t s);   // and launch_pack's work
void launch_column_sum(const ColumnSumArgs& a, hipStream_t s);

// Rows to codes of 8 bits, q[r, c] = x[r, c] ((1 / A) 127) rounded, and
// scale[r] = A / 127, with A the largest magnitude of row r.
struct QuantizeArgs {
  Mat x, q;
  int64_t rows, cols;
  float* scale;
};
hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t s);

// Forward products of codes of 8 bits: in GemmArgs, ld and K in elements for
// few rows and direct ones, else in pairs of them (lines of whole 16 bytes,
// zeros past the last k). launch_pack_int8: copies of such lines; here all
// sizes in elements.
enum Int8Kernel { kInt8Few, kInt8Direct, kInt8Tiles };
bool few_rows_int8(int64_t M, int64_t N, int64_t K, bool gated);
// Whether operands that are not aligned are taken as they are (kInt8Direct), and
// the bytes of partial sums that it needs then.
bool direct_int8(int64_t M, int64_t N, int64_t K, bool gated);
size_t direct_int8_bytes(int64_t M, int64_t N, int64_t K, bool gated);
hipError_t launch_pack_int8(const PackArgs& a, hipStream_t s);
hipError_t launch_gemm_int8(Int8Kernel kernel, GemmArgs a, void* partials, hipStream_t s);

// Rows offsets[g] ... offsets[g + 1] of a matrix of `rows` rows are group g's;
// `count` groups. An offset outside of [0, rows] counts as its nearer end.
struct Groups {
  const int32_t* offsets;
  int count;
  int rows;
};
// Products by group: rows of a with the group's part of b (`b_rows` rows of it);
// a.M is not looked at. partials: experts_partial_bytes.
size_t experts_partial_bytes(const Groups& g, int64_t N, int64_t K, bool gated, bool direct);
hipError_t launch_experts(const GemmArgs& a, const Groups& g, int64_t b_rows, void* partials, hipStream_t s);
// Whether the forward product takes the kernel for few rows.
bool few_rows_experts(const Groups& g, int64_t N, int64_t K, bool gated);
// Whether a product by group with `wide` rows of weights or columns of dx takes
// operands as they are (GemmArgs::direct), where they are not aligned.
bool direct_experts(const Groups& g, int64_t wide);
// dz of the groups' rows, and the sums over ranges of each group's rows:
// partials [experts_back_ranges][N].
int64_t experts_back_ranges(const Groups& g);
hipError_t launch_experts_act_back(const ActBackArgs& a, const Groups& g, hipStream_t s);
// The gradients, each where it is given: dx, a product by group; dw, for each
// group out [dw.M, dw.N] = the product over its rows; dbias [groups, N] from
// the ranges' sums. partials: experts_back_bytes, where dx is given.
size_t experts_back_bytes(const Groups& g, int64_t N, int64_t wide);
hipError_t launch_experts_back(const GemmArgs* dx, const GemmArgs* dw, const float* sums, int64_t N, const Mat& dbias,
                               const Groups& g, int64_t b_rows, void* partials, hipStream_t s);

}  // namespace taco
