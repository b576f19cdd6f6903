// What the 8-bit activation calls launch, without a GPU: their host code
// (a8.hip, compiled host-only) linked against the few HIP runtime functions
// below, which record each launch instead of making it. Kernels are named as
// the compiler registers them.
//
// Reads one call per line from standard input, "quant M K", "norm M K",
// "product M N K out", "pair M N K out" or "swiglu M N K" (out: f32 or bf16),
// makes it with aligned addresses that nothing dereferences, and prints
// "<status> <work bytes>" followed by one "| <kernel> <workgroups> <lanes>"
// for every launch.
#include "q4g64.h"

#include <cxxabi.h>
#include <hip/hip_runtime_api.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <iostream>
#include <map>
#include <sstream>
#include <string>
#include <vector>

namespace {

struct Launch {
  std::string kernel;
  unsigned grid, block;
};
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
std::vector<Launch> g_launches;
dim3 g_grid, g_block;

}  // namespace

extern "C" {

void** __hipRegisterFatBinary(const void*) {
  static void* handle = nullptr;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  int status = 0;
  char* plain = abi::__cxa_demangle(name, nullptr, nullptr, &status);
  names()[host] = status == 0 ? plain : name;
  free(plain);
}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
  g_grid = grid, g_block = block;
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = g_grid, *block = g_block, *lds = 0, *stream = nullptr;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
  g_launches.push_back({names()[f], grid.x, block.x});
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return ""; }
hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }

}  // extern "C"

int main() {
  char* const d = reinterpret_cast<char*>(uintptr_t(0x7e0000000000ull));
  uint8_t* const q = reinterpret_cast<uint8_t*>(d);
  float* const f = reinterpret_cast<float*>(d);
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    std::string op, out;
    int64_t M = 0, N = 0, K = 0;
    in >> op >> M;
    if (op != "quant" && op != "norm") in >> N;
    in >> K >> out;
    const int type = out == "bf16" ? Q4_BF16 : Q4_F32;
    const size_t work = op == "swiglu" ? qmm_a8_swiglu_work_bytes(M, N, K) : 0;
    int rc = -1000;
    g_launches.clear();
    if (op == "quant") rc = quant_rows_a8(d, Q4_F32, K, M, K, q, K, f, M, nullptr);
    else if (op == "norm") rc = rms_norm_rows(d, Q4_F32, K, nullptr, Q4_F32, 0, nullptr, 0, f, 1e-5f, M, K, d, Q4_F32, K, nullptr);
    else if (op == "product") rc = qmm_a8_fp8b(d, nullptr, N, K, q, K, f, M, M, d, type, N, nullptr);
    else if (op == "pair") rc = qmm_a8_fp8b(d, d, N, K, q, K, f, M, M, d, type, N, nullptr);
    else if (op == "swiglu") rc = qmm_a8_swiglu_a8(d, d, N, K, q, K, f, M, M, q, N, f, M, d, work, nullptr);
    printf("%d %zu", rc, work);
    for (const Launch& l : g_launches) printf("|%s|%u|%u", l.kernel.c_str(), l.grid, l.block);
    printf("\n");
  }
}
