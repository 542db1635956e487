// Host-side argument checks of the norm, dropout and few-row product calls,
// built together with the library sources under AddressSanitizer and
// UndefinedBehaviorSanitizer (host code only; no kernel is launched, no GPU is
// needed): invalid arguments, empty calls and sizes at and past the limits
// must return their documented status without undefined behaviour.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/mxfp4.h"

static int failures = 0;

static void expect(const char* what, int64_t got, int64_t want) {
  if (got != want) {
    fprintf(stderr, "%s: got %lld want %lld\n", what, (long long)got, (long long)want);
    ++failures;
  }
}

int main() {
  void* p = reinterpret_cast<void*>(4096);               // never dereferenced
  uint16_t* h = static_cast<uint16_t*>(p);
  uint8_t* b = static_cast<uint8_t*>(p);
  float* f = static_cast<float*>(p);
  uint16_t* h8 = reinterpret_cast<uint16_t*>(4096 + 8);
  const int64_t max = INT64_MAX, big = (int64_t)1 << 40;
  const fp4_dtype bf = FP4_BF16, bad = static_cast<fp4_dtype>(9);

  expect("dropout type", fp4_dropout(1, 8, p, bad, 8, nullptr, 0, 0.1f, 0, 0, h, 8, nullptr), FP4_EINVAL);
  expect("dropout p", fp4_dropout(1, 8, p, bf, 8, nullptr, 0, NAN, 0, 0, h, 8, nullptr), FP4_EINVAL);
  expect("dropout p inf", fp4_dropout(1, 8, p, bf, 8, nullptr, 0, INFINITY, 0, 0, h, 8, nullptr), FP4_EINVAL);
  expect("dropout huge rows", fp4_dropout(max, 8, p, bf, 8, nullptr, 0, 0.1f, 0, 0, h, 8, nullptr), FP4_ESHAPE);
  expect("dropout huge both", fp4_dropout(max, max, p, bf, max, nullptr, 0, 0.1f, 0, 0, h, max, nullptr), FP4_ESHAPE);
  expect("dropout negative", fp4_dropout(-1, 8, p, bf, 8, nullptr, 0, 0.1f, 0, 0, h, 8, nullptr), FP4_ESHAPE);
  expect("dropout ld", fp4_dropout(2, 8, p, bf, 7, nullptr, 0, 0.1f, 0, 0, h, 8, nullptr), FP4_ESHAPE);
  expect("dropout empty", fp4_dropout(0, max, nullptr, bf, max, nullptr, 0, 1.0f, 0, 0, nullptr, max, nullptr), FP4_OK);
  expect("dropout null", fp4_dropout(2, 8, p, bf, 8, nullptr, 0, 0.1f, 0, 0, nullptr, 8, nullptr), FP4_EINVAL);

  const auto norm = [&](int64_t t, int64_t d, int64_t ld, float eps, fp4_format fm, uint8_t* scales, uint16_t* gamma) {
    return fp4_rmsnorm_producer(t, d, p, bf, ld, nullptr, 0, gamma, eps, 0.1f, ~0ull, ~0ull, h, f, nullptr, fm, b, scales,
                                nullptr);
  };
  expect("norm format", norm(1, 32, 32, 1e-5f, static_cast<fp4_format>(7), b, h), FP4_EINVAL);
  expect("norm eps", norm(1, 32, 32, -0.0f, FP4_E4M3, b, h), FP4_EINVAL);
  expect("norm eps nan", norm(1, 32, 32, NAN, FP4_E4M3, b, h), FP4_EINVAL);
  expect("norm scales", norm(1, 32, 32, 1e-5f, FP4_E4M3, nullptr, h), FP4_EINVAL);
  expect("norm huge d", norm(1, max - 31, max - 31, 1e-5f, FP4_E4M3, b, h), FP4_ESHAPE);
  expect("norm huge t", norm(max, 32, 32, 1e-5f, FP4_E4M3, b, h), FP4_ESHAPE);
  expect("norm align", norm(1, 32, 32, 1e-5f, FP4_E4M3, b, h8), FP4_EALIGN);
  expect("norm empty", norm(0, 32, 32, 1e-5f, FP4_E4M3, b, nullptr), FP4_OK);

  expect("workspace", fp4_rmsnorm_backward_workspace(max, 32768), 512 * 32768 * 4);
  expect("workspace refused", fp4_rmsnorm_backward_workspace(1, max), -1);
  expect("workspace negative", fp4_rmsnorm_backward_workspace(INT64_MIN, 32), -1);
  const auto bwd = [&](int64_t t, int64_t d, void* ws, int64_t size) {
    return fp4_rmsnorm_backward(t, d, p, FP4_F32, d, h, d, f, h, nullptr, 0, 0.1f, 0, 0, h, h, f, 0, ws, size, nullptr);
  };
  expect("backward workspace", bwd(4, 64, p, 255), FP4_ESHAPE);
  expect("backward no workspace", bwd(4, 64, nullptr, 1 << 20), FP4_EINVAL);
  expect("backward huge t", bwd(max, 64, p, max), FP4_ESHAPE);
  expect("backward huge d", bwd(4, max, p, max), FP4_ESHAPE);
  expect("backward d 0", bwd(4, 0, nullptr, 0), FP4_OK);

  const auto mv = [&](int64_t m, int64_t n, int64_t k, int64_t ldx, int64_t ldc) {
    return fp4_matvec(m, n, k, p, ldx, nullptr, b, b, f, ldc, 0, nullptr);
  };
  expect("matvec m", mv(65, 16, 32, 32, 16), FP4_ESHAPE);
  expect("matvec m min", mv(INT64_MIN, 16, 32, 32, 16), FP4_ESHAPE);
  expect("matvec n", mv(1, max, 32, 32, max), FP4_ESHAPE);
  expect("matvec k", mv(1, 16, max - 31, max - 31, 16), FP4_ESHAPE);
  expect("matvec ldx", mv(64, 16, 32, big, 16), FP4_ESHAPE);
  expect("matvec ldc", mv(1, 16, 32, 32, 15), FP4_ESHAPE);
  expect("matvec empty", mv(0, max, 32, 32, max), FP4_OK);
  expect("nv stride", fp4_nv_matvec(1, 16, 32, h, 32, b, b, f, -1, f, 16, 0, nullptr), FP4_EINVAL);
  expect("nv null", fp4_nv_matvec(1, 16, 32, h, 32, b, b, nullptr, 0, f, 16, 0, nullptr), FP4_EINVAL);
  expect("swiglu f", fp4_swiglu_matvec(1, max, 32, p, 32, nullptr, b, b, h, nullptr), FP4_ESHAPE);
  expect("swiglu ldx", fp4_swiglu_matvec(1, 16, 32, p, 64, b, b, b, h, nullptr), FP4_ESHAPE);
  expect("swiglu empty", fp4_swiglu_matvec(0, 16, 32, nullptr, 32, nullptr, nullptr, nullptr, nullptr, nullptr), FP4_OK);

  printf("operator_checks: %d failure(s)\n", failures);
  return failures != 0;
}
