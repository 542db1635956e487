// The launches that the host code of the expert and epilogue calls decides on,
// recorded instead of made: the sources are included with the launch macro
// replaced, so that no kernel runs and no GPU is needed.  Reads one call a line
// from standard input and prints one line for it: the status, then "kernel grid.x
// grid.y grid.z block" for every launch.
//   ga   m n k                     fp4_gemm_act
//   mva  m n k ldx e4m3 offset     fp4_matvec_act (scales at `offset`)
//   ab   m n fp32 act bias         fp4_act_backward
//   sort t k experts align bytes   fp4_expert_sort
//   gat  t k d rows                fp4_expert_gather
//   com  t k d rows fp32           fp4_expert_combine
//   cob  t k d rows dy32 z32       fp4_expert_combine_backward
//   ge   experts rows n k          fp4_gemm_experts
//   gw   experts tokens m n        fp4_gemm_experts_wgrad
//   sw   experts rows f d          fp4_swiglu_producer_experts
//   mve  experts rows n k e4m3 offset   fp4_matvec_experts
//   sme  experts rows f d e4m3 offset   fp4_swiglu_matvec_experts
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

#include "../../precision_mxfp4_producers_amd/csrc/act.hip"
#include "../../precision_mxfp4_producers_amd/csrc/experts.hip"
#include "../../precision_mxfp4_producers_amd/csrc/gemm_act.hip"
#include "../../precision_mxfp4_producers_amd/csrc/gemm_experts.hip"
#include "../../precision_mxfp4_producers_amd/csrc/matvec_act.hip"
#include "../../precision_mxfp4_producers_amd/csrc/matvec_experts.hip"

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
  int32_t* const i = static_cast<int32_t*>(p);
  char line[256], op[16];
  const int64_t big = (int64_t)1 << 62;
  while (fgets(line, sizeof line, stdin)) {
    long long v[6] = {};
    if (sscanf(line, "%15s %lld %lld %lld %lld %lld %lld", op, v, v + 1, v + 2, v + 3, v + 4, v + 5) < 3) continue;
    launches.clear();
    int st = -1;
    const auto is = [&](const char* name) { return !strcmp(op, name); };
    const auto type = [](long long f32) { return f32 ? FP4_F32 : FP4_BF16; };
    if (is("ga")) st = fp4_gemm_act(v[0], v[1], v[2], b, b, b, b, p, FP4_BF16, FP4_ACT_GELU, h, v[1], h, p, FP4_BF16, v[1], nullptr);
    if (is("mva"))
      st = fp4_matvec_act(v[0], v[1], v[2], p, v[3], v[4] ? b : nullptr, b, b + v[5], p, FP4_BF16, FP4_ACT_GELU, h, v[1], p,
                          FP4_BF16, v[1], nullptr);
    if (is("ab"))
      st = fp4_act_backward(v[0], v[1], p, type(v[2]), v[1], h, v[1], (fp4_act)v[3], h, v[4] ? f : nullptr, 0, p, big, nullptr);
    if (is("sort")) st = fp4_expert_sort(v[0], v[1], v[2], p, (int)v[4], v[3], fp4_expert_capacity(v[0], v[1], v[2], v[3]), i, i, i, p, big, nullptr);
    if (is("gat")) st = fp4_expert_gather(v[0], v[1], v[2], v[3], h, v[2], i, h, FP4_E2M1, b, b, p, big, nullptr);
    if (is("com")) st = fp4_expert_combine(v[0], v[1], v[2], v[3], p, type(v[4]), v[2], i, f, h, v[2], h, v[2], nullptr);
    if (is("cob"))
      st = fp4_expert_combine_backward(v[0], v[1], v[2], v[3], p, type(v[4]), v[2], p, type(v[5]), v[2], i, i, f, h, f, nullptr);
    if (is("ge"))
      st = fp4_gemm_experts(v[0], v[1], v[2], v[3], i, b, b, b, b, nullptr, nullptr, nullptr, nullptr, p, FP4_F32, v[2], nullptr);
    if (is("gw")) st = fp4_gemm_experts_wgrad(v[0], v[1], v[2], v[3], i, b, b, b, b, p, FP4_F32, 0, nullptr);
    if (is("sw")) st = fp4_swiglu_producer_experts(v[0], v[1], v[2], v[3], i, b, b, b, b, h, h, b, b, b, b, 0, nullptr);
    if (is("mve"))
      st = fp4_matvec_experts(v[0], v[1], v[2], v[3], i, p, v[3], v[4] ? b : nullptr, b, b + v[5], f, v[2], nullptr);
    if (is("sme")) st = fp4_swiglu_matvec_experts(v[0], v[1], v[2], v[3], i, p, v[3], v[4] ? b : nullptr, b, b + v[5], h, nullptr);
    printf("%d%s\n", st, launches.c_str());
  }
  return 0;
}
