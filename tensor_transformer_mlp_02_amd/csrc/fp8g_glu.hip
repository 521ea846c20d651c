// The gated block's launches: fp32 sums, since the scales of its codes are
// fp32 results.
#include "fp8g_tile.h"

namespace tpmlp {
namespace g8 {

template <int SC, int FMT, int EPI>
static hipError_t launch_glu(G8GemmArgs& a, hipStream_t st) {
  const int64_t cols = EPI == G_GLU_FWD ? 128 : 256;
  const int64_t big = ((a.M + 255) / 256) * ((a.N + cols - 1) / cols);
  if (big >= 192) return launch<2, 4, 4, 2, SC, true, FMT, 0, SUM_F32, EPI>(a, st);
  // one group of columns a workgroup
  constexpr int FN = EPI == G_GLU_FWD ? 2 : 1;
  return launch<1, 8, FN, 3, SC, true, FMT, 0, SUM_F32, EPI>(a, st);
}

}  // namespace g8

hipError_t g8_glu_fwd_launch(int scale, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  return scale == TP_GROUP_F32 ? launch_glu<0, 0, G_GLU_FWD>(a, st) : launch_glu<1, 0, G_GLU_FWD>(a, st);
}

hipError_t g8_glu_bwd_launch(int fmt, int scale, G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (fmt == 0) return scale == TP_GROUP_F32 ? launch_glu<0, 0, G_GLU_BWD>(a, st) : launch_glu<1, 0, G_GLU_BWD>(a, st);
  return scale == TP_GROUP_F32 ? launch_glu<0, 1, G_GLU_BWD>(a, st) : launch_glu<1, 1, G_GLU_BWD>(a, st);
}

}  // namespace tpmlp
