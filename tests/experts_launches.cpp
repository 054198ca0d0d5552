// The launches of calls of the products by group, without a GPU: for each line
// "call groups M N K offset" of the standard input, with call one of
//   linear gated             forward
//   linear-dx linear-dw linear-both linear-db linear-all   gated-dx gated-dw gated-both   gradients
// and every array `offset` elements (and its rows `offset` elements) off 16
// bytes, the entry point's status and after it each launch that it makes, as
// "kernel|grid x|grid y|threads of a workgroup|bytes of LDS", on one line. The entry points
// and their plans are the library's own; the arrays are addresses that nothing
// reads, and a workspace is as large as its *_workspace_bytes says.
#include <cxxabi.h>
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <string>
#include <typeinfo>

static std::string launches;
template <auto K>
struct Name {};
template <auto K>
static void record(dim3 grid, dim3 block, size_t lds) {
  char* text = abi::__cxa_demangle(typeid(Name<K>).name(), nullptr, nullptr, nullptr);
  std::string name = text;
  free(text);
  name = name.substr(name.find("k_"));
  name = name.substr(0, name.find('('));   // without its arguments
  char sizes[96];
  snprintf(sizes, sizeof(sizes), "|%u|%u|%u|%zu", grid.x, grid.y, block.x, lds);
  launches += "\t" + name + sizes;
}
#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) record<kernel>(grid, block, lds)
#define hipGetLastError() hipSuccess

#include "../quantized_compression_tensor_amd/csrc_layers/experts.hip"
#include "../quantized_compression_tensor_amd/csrc_layers/experts_abi.hip"

namespace taco {
void launch_column_sum(const ColumnSumArgs&, hipStream_t) {}   // never called
hipError_t launch_pack(const PackArgs&, hipStream_t) { return launches += "\tpack|0|0|0|0", hipSuccess; }
hipError_t launch_act_back(const ActBackArgs&, const PackArgs&, hipStream_t) {
  return launches += "\tact_back|0|0|0|0", hipSuccess;
}
}  // namespace taco

static char* next_address;
static taco_array array(int64_t rows, int64_t cols, int32_t dtype, int64_t offset) {
  const int64_t stride = cols + offset, bytes = dtype == TACO_BF16 ? 2 : 4;
  const taco_array a = {next_address + offset * bytes, stride, dtype, 0};
  next_address += (rows * stride * bytes / 4096 + 2) * 4096;
  return a;
}

int main() {
  char call[32];
  long long groups, M, N, K, offset;
  while (scanf("%31s %lld %lld %lld %lld %lld", call, &groups, &M, &N, &K, &offset) == 6) {
    const std::string what = call;
    const bool gated = what.rfind("gated", 0) == 0;
    const int64_t wide = gated ? 2 * N : N;
    auto ends = [&](const char* s) { return what.size() > strlen(s) && what.substr(what.size() - strlen(s)) == s; };
    auto wants = [&](const char* s) { return ends(s) || (ends("-both") && strcmp(s, "-db")) || ends("-all"); };
    next_address = reinterpret_cast<char*>(int64_t(1) << 44);
    launches.clear();
    const taco_array none = {nullptr, 0, TACO_F32, 0};
    const taco_array x = array(M, K, TACO_BF16, offset), w = array(groups * wide, K, TACO_BF16, offset);
    const taco_array y = array(M, N, TACO_BF16, offset), z = array(M, wide, TACO_BF16, offset);
    const taco_array dx = array(M, K, TACO_BF16, offset), dw = array(groups * wide, K, TACO_BF16, offset);
    const taco_array db = array(groups, N, TACO_F32, 0);
    const int32_t* o = static_cast<const int32_t*>(array(groups + 1, 1, TACO_F32, 0).data);
    void* ws = next_address;
    int st;
    if (what == "linear") {
      st = taco_grouped_linear(x, w, none, TACO_ACT_GELU, o, (int)groups, y, z, M, N, K, ws,
                               taco_grouped_linear_workspace_bytes((int)groups, M, N, K), nullptr);
    } else if (what == "gated") {
      st = taco_grouped_gated_linear(x, w, TACO_ACT_SILU, o, (int)groups, y, z, M, N, K, ws,
                                     taco_grouped_gated_linear_workspace_bytes((int)groups, M, N, K), nullptr);
    } else if (gated) {
      st = taco_grouped_gated_linear_backward(y, x, w, TACO_ACT_SILU, z, o, (int)groups, wants("-dx") ? dx : none,
                                              wants("-dw") ? dw : none, M, N, K, ws,
                                              taco_grouped_gated_linear_backward_workspace_bytes((int)groups, M, N, K),
                                              nullptr);
    } else {
      st = taco_grouped_linear_backward(y, x, w, TACO_ACT_GELU, z, o, (int)groups, wants("-dx") ? dx : none,
                                        wants("-dw") ? dw : none, wants("-db") ? db : none, M, N, K, ws,
                                        taco_grouped_linear_backward_workspace_bytes((int)groups, M, N, K), nullptr);
    }
    printf("%d%s\n", st, launches.c_str());
  }
  return 0;
}
