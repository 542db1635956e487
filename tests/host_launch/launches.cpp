// The launches that the host code of the norm, dropout and few-row product
// calls decides on, recorded instead of made: the sources are included with
// the launch macro replaced, so that no kernel runs and no GPU is needed.
// Reads one call a line from standard input and prints one line for it: the
// status, then "kernel grid.x grid.y grid.z block" for every launch.
//   mv  m n k ldx e4m3 scales_offset     fp4_matvec
//   nv  m n k ldx scales_offset          fp4_nv_matvec
//   sw  m f d ldx e4m3 scales_offset     fp4_swiglu_matvec
//   norm t d fp32 residual               fp4_rmsnorm_producer
//   bwd t d fp32 ds                      fp4_rmsnorm_backward
//   drop rows cols fp32 residual         fp4_dropout
#include <cxxabi.h>
#include <dlfcn.h>
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <string>

static std::string launches;

static void record(const void* kernel, dim3 grid, dim3 block) {
  Dl_info info{};
  const char* name = dladdr(kernel, &info) && info.dli_sname ? info.dli_sname : "?";
  char* plain = abi::__cxa_demangle(name, nullptr, nullptr, nullptr);
  std::string s = plain ? plain : name;
  free(plain);
  if (s.rfind("void ", 0) == 0) s = s.substr(5);
  const size_t stub = s.find("__device_stub__");
  if (stub != std::string::npos) s = s.substr(stub + strlen("__device_stub__"));
  std::string id;
  for (const char c : s.substr(0, s.find('(')))
    if (c != ' ') id += c;
  launches += " " + id + " " + std::to_string(grid.x) + " " + std::to_string(grid.y) + " " + std::to_string(grid.z) + " " +
              std::to_string(block.x * block.y * block.z);
}

#undef hipLaunchKernelGGL
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  record(reinterpret_cast<const void*>(kernel), grid, block)
#define hipGetLastError() hipSuccess

#include "../../precision_mxfp4_producers_amd/csrc/matvec.hip"
#include "../../precision_mxfp4_producers_amd/csrc/norm.hip"

namespace mx { thread_local int g_last_hip_error = 0; }

// Host code only: the device code's image is absent and nothing registers it.
extern "C" {
void** __hipRegisterFatBinary(const void*) { return nullptr; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
}

int main() {
  void* const p = reinterpret_cast<void*>(4096);         // never dereferenced
  uint16_t* const h = static_cast<uint16_t*>(p);
  uint8_t* const b = static_cast<uint8_t*>(p);
  float* const f = static_cast<float*>(p);
  char line[256], op[16];
  while (fgets(line, sizeof line, stdin)) {
    long long v[6] = {};
    if (sscanf(line, "%15s %lld %lld %lld %lld %lld %lld", op, v, v + 1, v + 2, v + 3, v + 4, v + 5) < 3) continue;
    launches.clear();
    int st = -1;
    const fp4_dtype type = v[2] ? FP4_F32 : FP4_BF16;
    if (!strcmp(op, "mv")) st = fp4_matvec(v[0], v[1], v[2], p, v[3], v[4] ? b : nullptr, b, b + v[5], f, v[1], 0, nullptr);
    if (!strcmp(op, "nv")) st = fp4_nv_matvec(v[0], v[1], v[2], h, v[3], b, b + v[4], f, 0, f, v[1], 0, nullptr);
    if (!strcmp(op, "sw")) st = fp4_swiglu_matvec(v[0], v[1], v[2], p, v[3], v[4] ? b : nullptr, b, b + v[5], h, nullptr);
    if (!strcmp(op, "norm"))
      st = fp4_rmsnorm_producer(v[0], v[1], p, type, v[1], v[3] ? h : nullptr, v[1], h, 1e-5f, 0.1f, 1, 2, h, f, nullptr,
                                FP4_E4M3, b, b, nullptr);
    if (!strcmp(op, "bwd"))
      st = fp4_rmsnorm_backward(v[0], v[1], p, type, v[1], h, v[1], f, h, v[3] ? h : nullptr, v[1], 0.1f, 1, 2, h, h, f, 0, p,
                                fp4_rmsnorm_backward_workspace(v[0], v[1]), nullptr);
    if (!strcmp(op, "drop"))
      st = fp4_dropout(v[0], v[1], p, type, v[1], v[3] ? h : nullptr, v[1], 0.1f, 1, 2, h, v[1], nullptr);
    printf("%d%s\n", st, launches.c_str());
  }
  return 0;
}
