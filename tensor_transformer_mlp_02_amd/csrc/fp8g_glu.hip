// The gated block's launches: fp32 sums, since its scales and codes are made from the fp32
// values.  4096 tokens, 8192 -> 3584: forward 404 to 420 us (1.17 PFLOP/s), backward 245; with E8M0 scales 390, 237.
#include "fp8g_tile.h"

namespace tpmlp {
namespace g8 {

template <int SC, int FMT, int EPI>
static hipError_t launch_glu(G8Form form, G8GemmArgs& a, hipStream_t st) {
  constexpr int RAW = EPI == G_GLU_FWD ? G_RAW_FWD : G_RAW_BWD, FN = EPI == G_GLU_FWD ? 2 : 1;
  switch (form) {
    case G8_LARGE: return launch<2, 4, 8, 4, 2, SC, true, FMT, 0, SUM_F32, EPI>(a, st);
    case G8_GROUP: return launch<1, 8, 8, FN, 3, SC, true, FMT, 0, SUM_F32, EPI>(a, st);
    case G8_SMALL: return launch<1, 4, 4, 2, 3, SC, true, FMT, 0, SUM_F32, RAW>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace g8

hipError_t g8_glu_fwd_launch(G8Form form, int scale, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  return scale == TP_GROUP_F32 ? launch_glu<0, 0, G_GLU_FWD>(form, a, st) : launch_glu<1, 0, G_GLU_FWD>(form, a, st);
}

hipError_t g8_glu_bwd_launch(G8Form form, int fmt, int scale, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (fmt == 0) return scale == TP_GROUP_F32 ? launch_glu<0, 0, G_GLU_BWD>(form, a, st) : launch_glu<1, 0, G_GLU_BWD>(form, a, st);
  return scale == TP_GROUP_F32 ? launch_glu<0, 1, G_GLU_BWD>(form, a, st) : launch_glu<1, 1, G_GLU_BWD>(form, a, st);
}

}  // namespace tpmlp
