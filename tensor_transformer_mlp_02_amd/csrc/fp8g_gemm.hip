// The product with bf16 results: its rounding is some 100 times what the FP8
// instruction loses in a group's sum, so that instruction adds the products.
#include "fp8g_tile.h"

namespace tpmlp {
namespace g8 {

template <int SC, bool SQ, int FMT_A, int FMT_B>
static hipError_t launch_plain(G8GemmArgs& a, hipStream_t st) {
  const int64_t big = ((a.M + 255) / 256) * ((a.N + 255) / 256);
  // (fp32 scales for each column: no registers for them beside a large tile's sums)
  if constexpr (SC == TP_GROUP_E8M0 || SQ) {
    if (big >= 192) return launch<2, 4, 4, 2, SC, SQ, FMT_A, FMT_B, SUM_FP8, G_STORE>(a, st);
  }
  return launch<1, 4, 2, 4, SC, SQ, FMT_A, FMT_B, SUM_FP8, G_STORE>(a, st);
}
template <int SC, bool SQ>
static hipError_t launch_formats(int fa, int fb, G8GemmArgs& a, hipStream_t st) {
  if (fa == 0 && fb == 0) return launch_plain<SC, SQ, 0, 0>(a, st);
  if (fa == 1 && fb == 0) return launch_plain<SC, SQ, 1, 0>(a, st);
  if (fa == 0 && fb == 1) return launch_plain<SC, SQ, 0, 1>(a, st);
  return hipErrorInvalidValue;
}

}  // namespace g8

hipError_t g8_gemm_bf16_launch(int fmt_a, int fmt_b, int scale, int square, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (scale == TP_GROUP_F32)
    return square ? launch_formats<0, true>(fmt_a, fmt_b, a, st) : launch_formats<0, false>(fmt_a, fmt_b, a, st);
  return square ? launch_formats<1, true>(fmt_a, fmt_b, a, st) : launch_formats<1, false>(fmt_a, fmt_b, a, st);
}

}  // namespace tpmlp
