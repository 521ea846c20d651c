// The argument checks of include/tpmlp_fp8g.h under AddressSanitizer and
// UndefinedBehaviorSanitizer: 20000 seeded fuzzed calls (descriptors, sizes,
// NULL / misaligned / overlapping pointers), and the choice of a kernel over its whole range of
// sizes.  There is no GPU: every call has to end in an error status with a message, and none may
// reach a launcher.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <random>

#include "fp8g.h"
#include "launch.h"

namespace tpmlp {
[[noreturn]] static void reached(const char* what) {
  fprintf(stderr, "a call reached %s\n", what);
  exit(3);
}
hipError_t gemm_bf16(GemmKind, GemmArgs&, hipStream_t) { reached("gemm_bf16"); }
hipError_t gemm_f32(GemmKind, GemmArgs&, hipStream_t) { reached("gemm_f32"); }
hipError_t gemm_fp8(GemmKind, GemmArgs&, hipStream_t) { reached("gemm_fp8"); }
hipError_t partial_sum_launch(int, int, const void* const*, int64_t, void*, int, hipStream_t) { reached("partial_sum"); }
hipError_t fp8_quantize_launch(int, bool, int64_t, int64_t, const void*, const float*, void*, float*, hipStream_t) { reached("fp8_quantize"); }
hipError_t zero_float_launch(float*, hipStream_t) { reached("zero_float"); }
hipError_t fp8_scale_update_launch(int, int, int, int, float*, float*, float*, float*, hipStream_t) { reached("scale_update"); }
hipError_t byte_transpose_launch(int64_t, int64_t, const void*, void*, hipStream_t) { reached("byte_transpose"); }
hipError_t moe_permute_launch(int, const int32_t*, int64_t, int64_t, int64_t, const void*, void*, hipStream_t) { reached("permute"); }
hipError_t moe_combine_launch(int, const int32_t*, const int32_t*, const float*, int64_t, int64_t, int64_t, const void*, void*, hipStream_t) { reached("combine"); }
hipError_t moe_combine_bwd_launch(int, const int32_t*, const float*, int64_t, int64_t, int64_t, const void*, const void*, void*, float*, hipStream_t) { reached("combine_bwd"); }
hipError_t g8_quant_launch(int, int, int, int, const G8QuantArgs&, hipStream_t) { reached("quant"); }
hipError_t g8_gemm_bf16_launch(bool, int, int, int, int, G8GemmArgs&, hipStream_t) { reached("gemm bf16"); }
hipError_t g8_gemm_f32_launch(bool, int, int, int, int, G8GemmArgs&, hipStream_t) { reached("gemm f32"); }
hipError_t g8_glu_fwd_launch(G8Form, int, G8GemmArgs&, hipStream_t) { reached("glu_fwd"); }
hipError_t g8_glu_bwd_launch(G8Form, int, int, G8GemmArgs&, hipStream_t) { reached("glu_bwd"); }
hipError_t g8_gemm_few_launch(int, int, int, int, const G8GemmArgs&, hipStream_t) { reached("gemm few"); }
hipError_t g8_glu_fwd_few_launch(int, const G8GemmArgs&, hipStream_t) { reached("glu_fwd few"); }
hipError_t g8_glu_bwd_few_launch(int, int, const G8GemmArgs&, hipStream_t) { reached("glu_bwd few"); }
}  // namespace tpmlp

static std::mt19937_64 rng(20240917);
static uint64_t below(uint64_t n) { return rng() % n; }
template <typename T>
static T pick(std::initializer_list<T> v) { return v.begin()[below(v.size())]; }

static void* pointer() {
  switch (below(12)) {
    case 0: return nullptr;
    case 1: return (void*)(uintptr_t)(1 + below(64));
    case 2: return (void*)(UINT64_MAX - below(4096));
    case 3: return (void*)(((uintptr_t)1 << 44) + below(1 << 20));
    default: return (void*)(((uintptr_t)(1 + below(60)) << 40) & ~(uintptr_t)15);
  }
}
static int64_t size() {
  return pick<int64_t>({0, 1, 7, 8, 128, 256, 1000, 4096, -1, INT64_MIN, INT64_MAX, (int64_t)1 << 30, ((int64_t)1 << 30) + 1,
                        (int64_t)1 << 21, (int64_t)1 << 40, (int64_t)below(5000), (int64_t)below(40) * 8, (int64_t)below(40) * 128});
}
static int32_t small() { return pick<int32_t>({0, 1, 2, -1, INT32_MIN, INT32_MAX, (int32_t)below(4)}); }
static int32_t flag() { return below(12) ? (int32_t)below(2) : small(); }
static void* there() { return below(8) ? (void*)((uintptr_t)(1 + below(4000)) << 36) : pointer(); }

int main() {
  using namespace tpmlp;
  long seen = 0;
  for (int it = 0; it < 20000; ++it) {
    int rc;
    switch (below(4)) {
      case 0: {
        tp_fp8g_quant_desc d{size(), size(), flag(), flag(), flag(), flag()};
        if (below(3)) d.rows = (int64_t)below(3000), d.cols = 8 * (int64_t)(1 + below(300));
        rc = tp_fp8g_quantize(below(50) ? &d : nullptr, there(), there(), there(), there(), there(), nullptr);
        break;
      }
      case 1: {
        tp_fp8g_gemm_desc d{size(), size(), size(), 1, flag(), flag(), flag(), flag(), flag(), flag()};
        if (below(3)) d.M = (int64_t)below(3000), d.N = 8 * (int64_t)(1 + below(300)), d.K = 128 * (int64_t)(1 + below(60));
        if (below(3)) d.accumulate = 0;
        if (below(3) == 0) d.parts = 2;
        if (below(20) == 0) d.parts = small();
        const bool two = d.parts == 2 || below(20) == 0;
        rc = tp_fp8g_gemm(below(50) ? &d : nullptr, there(), there(), there(), there(), two ? there() : nullptr,
                          two ? there() : nullptr, there(), nullptr);
        break;
      }
      default: {
        tp_fp8g_glu_desc d{size(), size(), size(), flag(), flag(), below(2) ? 0 : flag()};
        if (below(3)) d.N = (int64_t)below(3000), d.H = 8 * (int64_t)(1 + below(300)), d.F = 8 * (int64_t)(1 + below(300));
        const tp_fp8g_glu_desc* p = below(50) ? &d : nullptr;
        const size_t need = below(2) ? tp_fp8g_glu_fwd_workspace(p) : tp_fp8g_glu_bwd_workspace(p);
        const size_t ws = below(3) ? SIZE_MAX : need - (size_t)below(2);
        if (below(2))
          rc = tp_fp8g_glu_fwd(p, there(), there(), there(), there(), there(), there(), there(), there(), there(), there(),
                               there(), there(), there(), ws, nullptr);
        else
          rc = tp_fp8g_glu_bwd(p, there(), there(), there(), there(), there(), there(), there(), there(), there(), there(), ws,
                               nullptr);
        break;
      }
    }
    if (rc < 1 || rc > 8 || strlen(tp_last_error()) == 0) {
      fprintf(stderr, "call %d: status %d, message \"%s\"\n", it, rc, tp_last_error());
      return 2;
    }
    seen |= 1L << rc;
  }
  // every kind of refusal has been met
  for (int k : {TP_ERR_NULL, TP_ERR_SHAPE, TP_ERR_DTYPE, TP_ERR_ALIGN, TP_ERR_WORKSPACE, TP_ERR_DEVICE, TP_ERR_ALIAS})
    if (!(seen >> k & 1)) {
      fprintf(stderr, "no call ended with status %d\n", k);
      return 4;
    }
  // the choice of a kernel, at the ends of its range and between
  const int64_t dims[] = {1, 64, 65, 333, 4096, (int64_t)1 << 21, (int64_t)1 << 30};
  for (int64_t M : dims)
    for (int64_t N : {(int64_t)8, (int64_t)1000, (int64_t)1 << 21})
      for (int64_t kt : {1, 28, 16384}) {
        for (int f = 0; f < 4; ++f) {
          const G8Form g = g8_plan_gemm(M, N, kt, f & 1, f & 2);
          if (g == G8_GROUP || (g == G8_LARGE && !(f & 2)) || (M <= 64 && g != G8_FEW)) return 5;
        }
        for (int back = 0; back < 2; ++back)
          if (M <= 64 && g8_plan_glu(M, N, kt, back) != G8_FEW) return 6;
      }
  printf("OK\n");
  return 0;
}
