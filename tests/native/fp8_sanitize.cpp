// Host-only driver of the argument checks of the 8-bit entry points
// (rotated_bit_amd/csrc/validate.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_fp8_sanitized.py: every field and
// argument at extreme values, alone and in pairs.  Pointers are stand-in
// addresses that are never dereferenced.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "../../rotated_bit_amd/csrc/validate.hpp"

using namespace harp;

static const int32_t kInts[] = {std::numeric_limits<int32_t>::min(),
                                -1,
                                0,
                                1,
                                15,
                                16,
                                17,
                                32768,
                                32769,
                                65536,
                                65537,
                                262144,
                                262145,
                                std::numeric_limits<int32_t>::max()};
static const float kFloats[] = {-1.0f, 0.0f, 1e-6f, NAN, INFINITY, -INFINITY, 3e38f};

int main() {
  const void* const A = reinterpret_cast<const void*>(uintptr_t{0x10000});
  long ok = 0, all = 0;
  const auto count = [&](harp_status s) {
    ++all;
    ok += s == HARP_OK;
  };
  for (int32_t m : kInts)
    for (int32_t d : kInts) {
      for (float eps : kFloats)
        for (bool fp8 : {false, true})
          for (int dt : {-1, 0, 1, 2, 0x7fffffff})
            count(validate_rmsnorm(A, dt & 1, A, A, A, 0, eps, A, dt, fp8, A, m, d));
      count(validate_silu_mul_fp8(A, 1, A, A, m, d));
      for (int32_t k : kInts)
        for (int32_t e : kInts) {
          harp_fp8_weight w{};
          w.N = d;
          w.K = k;
          w.experts = e;
          w.w = static_cast<const uint8_t*>(A);
          w.scale = static_cast<const float*>(A);
          count(validate_fp8_gemm(&w, A, A, A, 0, m));
          for (int32_t r : kInts)
            for (const void* rows : {static_cast<const void*>(nullptr), A})
              count(validate_fp8_gemm_grouped(&w, A, A, r, rows, A, A, 1, m));
        }
    }
  if (validate_fp8_gemm(nullptr, A, A, A, 0, 1) != HARP_ERR_NULL || ok == 0 || ok == all) {
    std::fprintf(stderr, "%ld of %ld accepted\n", ok, all);
    return 1;
  }
  std::printf("all checks passed (%ld of %ld accepted)\n", ok, all);
  return 0;
}
