// The product with bf16 results: its rounding is some 100 times what the FP8
// instruction loses in a group's sum, so that instruction adds the products
// (4096 x 8192 x 3584: 119 us, and 206 with fp32 sums).
#include "fp8g_tile.h"

namespace tpmlp {
namespace g8 {

template <int SC, bool SQ, int FMT_A, int FMT_B>
static hipError_t launch_plain(bool large, G8GemmArgs& a, hipStream_t st) {
  // (fp32 scales for each column: no registers for them beside a large tile's sums)
  if constexpr (SC == TP_GROUP_E8M0 || SQ) {
    if (large) return launch<2, 4, 8, 4, 2, SC, SQ, FMT_A, FMT_B, SUM_FP8, G_STORE>(a, st);
  }
  return launch<1, 4, 4, 2, 3, SC, SQ, FMT_A, FMT_B, SUM_FP8, G_STORE>(a, st);
}
template <int SC, bool SQ>
static hipError_t launch_formats(bool large, int fa, int fb, G8GemmArgs& a, hipStream_t st) {
  if (fa == 0 && fb == 0) return launch_plain<SC, SQ, 0, 0>(large, a, st);
  if (fa == 1 && fb == 0) return launch_plain<SC, SQ, 1, 0>(large, a, st);
  if (fa == 0 && fb == 1) return launch_plain<SC, SQ, 0, 1>(large, a, st);
  return hipErrorInvalidValue;
}

}  // namespace g8

hipError_t g8_gemm_bf16_launch(bool large, int fa, int fb, int scale, int square, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (scale == TP_GROUP_F32)
    return square ? launch_formats<0, true>(large, fa, fb, a, st) : launch_formats<0, false>(large, fa, fb, a, st);
  return square ? launch_formats<1, true>(large, fa, fb, a, st) : launch_formats<1, false>(large, fa, fb, a, st);
}

}  // namespace tpmlp
