// The product with fp32 results: codes widened to bf16, fp32 sums.
// 8192 x 3584 x 4096 with E8M0 scales, added into C: 227 to 240 us, of them 30 for C; with an fp32 scale for
// each column, which has the 64 x 128 tile alone, 343.
#include "fp8g_tile.h"

namespace tpmlp {
namespace g8 {

template <int SC, bool SQ, int FMT_A, int FMT_B>
static hipError_t launch_plain(bool large, G8GemmArgs& a, hipStream_t st) {
  // (fp32 scales for each column: no registers for them beside a large tile's sums)
  if constexpr (SC == TP_GROUP_E8M0 || SQ) {
    if (large) return launch<2, 4, 8, 4, 2, SC, SQ, FMT_A, FMT_B, SUM_F32, G_STORE>(a, st);
  }
  return launch<1, 4, 4, 2, 3, SC, SQ, FMT_A, FMT_B, SUM_F32, G_STORE>(a, st);
}
template <int SC, bool SQ>
static hipError_t launch_formats(bool large, int fa, int fb, G8GemmArgs& a, hipStream_t st) {
  if (fa == 0 && fb == 0) return launch_plain<SC, SQ, 0, 0>(large, a, st);
  if (fa == 1 && fb == 0) return launch_plain<SC, SQ, 1, 0>(large, a, st);
  if (fa == 0 && fb == 1) return launch_plain<SC, SQ, 0, 1>(large, a, st);
  return hipErrorInvalidValue;
}

}  // namespace g8

hipError_t g8_gemm_f32_launch(bool large, int fa, int fb, int scale, int square, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (scale == TP_GROUP_F32)
    return square ? launch_formats<0, true>(large, fa, fb, a, st) : launch_formats<0, false>(large, fa, fb, a, st);
  return square ? launch_formats<1, true>(large, fa, fb, a, st) : launch_formats<1, false>(large, fa, fb, a, st);
}

}  // namespace tpmlp
