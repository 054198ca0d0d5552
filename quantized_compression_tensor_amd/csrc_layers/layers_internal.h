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
};

// Workgroups of the norm's backward pass: two for each CU of the device. Each
// adds up the weight's gradient over its rows and writes one partial sum per
// column, so their number is also what the workspace holds.
constexpr int kNormBackGroups = 512;

struct NormBackArgs {
  Mat dy, x, weight, dx, dweight, dbias;
  int64_t rows;
  int cols;
  const float *mean, *rstd;
  float* partials;      // [groups][2][cols]
};

int norm_back_groups(int64_t rows, int64_t cols);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_back(const NormBackArgs& a, hipStream_t s);

}  // namespace taco
