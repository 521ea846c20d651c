// The argument checks of include/tpmlp_block.h under AddressSanitizer and
// UndefinedBehaviorSanitizer: 20000 seeded fuzzed calls (descriptors, sizes,
// NULL / misaligned / overlapping pointers, tensor tables).  There is no GPU:
// every call has to end in an error status with a message, and none may reach
// a launcher.
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <random>
#include <vector>

#include "block_launch.h"
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
hipError_t norm_fwd_launch(int, int, const NormFwdArgs&, hipStream_t) { reached("norm_fwd"); }
hipError_t norm_bwd_launch(int, int, NormBwdArgs&, hipStream_t) { reached("norm_bwd"); }
size_t norm_bwd_workspace(const tp_norm_desc& d) { return (size_t)d.H * 16 + (size_t)d.N * 8; }
hipError_t route_fwd_launch(const tp_route_desc&, const void*, const float*, int32_t*, float*, hipStream_t) { reached("route_fwd"); }
hipError_t route_bwd_launch(const tp_route_desc&, const void*, const int32_t*, const float*, const int32_t*, int64_t, void*, hipStream_t) { reached("route_bwd"); }
size_t route_tables_workspace(int64_t N, int K, int n_local) { return (size_t)(N * K / 256 + 1) * ((size_t)n_local + 1) * 4; }
hipError_t route_tables_launch(const TablesArgs&, hipStream_t) { reached("tables"); }
hipError_t adamw_launch(const tp_adamw_desc&, int, const tp_adamw_tensor*, const int32_t*, const float*, const float*, hipStream_t) { reached("adamw"); }
}  // namespace tpmlp

static std::mt19937_64 rng(20240607);
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
  return pick<int64_t>({0, 1, 2, 7, 8, 64, 100, 4096, -1, INT64_MIN, INT64_MAX, (int64_t)1 << 30,
                        ((int64_t)1 << 30) + 1, (int64_t)1 << 21, (int64_t)1 << 40, (int64_t)below(5000)});
}
static int32_t small() {
  return pick<int32_t>({0, 1, 2, 3, 8, 64, 65, 1024, 1025, -1, INT32_MIN, INT32_MAX, (int32_t)below(70)});
}
static float real() { return pick<float>({0.f, 1.f, -1.f, 1e-5f, INFINITY, NAN, 1e-40f, 3e38f}); }

int main() {
  long seen = 0;
  for (int it = 0; it < 20000; ++it) {
    int rc = 0;
    switch (below(6)) {
      case 0:
      case 1: {
        tp_norm_desc d{size(), size(), size(), pick({0, 1, 0, 1, small()}), pick({0, 1, 0, 1, small()}), real(), real(), real()};
        if (below(2)) d = tp_norm_desc{12, 64, (int64_t)below(4), (int)below(2), (int)below(2), 1e-5f, 1.f, 1.f};
        const tp_norm_desc* p = below(50) ? &d : nullptr;
        void* v[18];
        for (auto& x : v) x = pointer();
        if (below(2))
          rc = tp_block_norm_fwd(p, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], (float*)v[9], (float*)v[10], nullptr);
        else
          rc = tp_block_norm_bwd(p, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], (float*)v[8], (float*)v[9], v[10], v[11],
                                 (float*)v[12], (float*)v[13], (float*)v[14], (float*)v[15], (float*)v[16], v[17],
                                 below(2) ? SIZE_MAX : (size_t)below(10000), (int)below(3), nullptr);
        (void)tp_block_norm_bwd_workspace(p);
        break;
      }
      case 2:
      case 3: {
        tp_route_desc d{size(), small(), small(), small(), small(), small(), small(), small(), small(), real()};
        if (below(2)) d = tp_route_desc{10, 64, (int)below(9), 8, (int)below(9), (int)below(3), (int)below(2), (int)below(2), (int)below(2), 1.f};
        const tp_route_desc* p = below(50) ? &d : nullptr;
        if (below(2))
          rc = tp_moe_route_fwd(p, pointer(), (float*)pointer(), (int32_t*)pointer(), (float*)pointer(), nullptr);
        else
          rc = tp_moe_route_bwd(p, pointer(), (int32_t*)pointer(), (float*)pointer(), (int32_t*)pointer(), size(), pointer(), nullptr);
        break;
      }
      case 4: {
        const int64_t N = below(2) ? 10 : size();
        const int32_t K = below(2) ? 4 : small(), L = below(2) ? 16 : small();
        rc = tp_moe_route_tables(N, K, small(), L, below(2) ? 40 : size(), (int32_t*)pointer(), (float*)pointer(),
                                 (int32_t*)pointer(), (int32_t*)pointer(), (float*)pointer(), (int32_t*)pointer(),
                                 (int32_t*)pointer(), (int32_t*)pointer(), pointer(), below(2) ? SIZE_MAX : (size_t)below(5000), nullptr);
        (void)tp_moe_route_tables_workspace(N, K, L);
        break;
      }
      default: {
        tp_adamw_desc d{pick<double>({1e-3, 0.0, -1.0, INFINITY, NAN}), pick<double>({0.9, 0.0, 1.0, NAN, -1.0}),
                        pick<double>({0.95, 0.0, 1.0, NAN}), pick<double>({1e-8, 0.0, 1e-40, INFINITY}), small(), small(),
                        pick({8, 32, small()}), (uint32_t)rng()};
        if (below(4)) d = tp_adamw_desc{1e-3, 0.9, 0.95, 1e-8, 1, (int)below(2), below(2) ? 8 : 32, 1};
        std::vector<tp_adamw_tensor> t(below(6));
        for (auto& x : t) {
          x = tp_adamw_tensor{(float*)pointer(), pointer(), pointer(), pointer(), pointer(), nullptr, nullptr,
                              below(2) ? (int64_t)below(5000) : size(), below(8) ? 0.1f : real(), below(20) ? 0 : small()};
          if (d.state_bits == 8 || below(10) == 0) {
            x.m_scale = (float*)pointer();
            x.v_scale = (float*)pointer();
          }
        }
        const int32_t n = below(20) ? (int32_t)t.size() : pick({-1, 65537, INT32_MIN});
        rc = tp_adamw_step(below(50) ? &d : nullptr, n, below(20) || t.empty() ? t.data() : nullptr,
                           below(3) ? nullptr : (int32_t*)pointer(), below(3) ? nullptr : (float*)pointer(),
                           below(3) ? nullptr : (float*)pointer(), nullptr);
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
  printf("OK\n");
  return 0;
}
