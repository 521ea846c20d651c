// Products of 8-bit codes with group scales for few rows, or few outputs
// behind a long sum.  A generated token's product is bound by the weights'
// bytes: each is read once, straight into registers, by the wavefront that multiplies it.
//
// A workgroup has up to 64 rows of A and 16 or 32 of the weight (the gated
// forward: 16 of both), and its four wavefronts deal the groups of the summed index among
// themselves: wavefront w takes groups w, w + 4, ...  Codes are widened to bf16
// for v_mfma_f32_16x16x32_bf16 with the weights first; lane (p = lane % 16, q = lane / 16)
// gives row p's codes 32 q .. + 31 of the group (32 bytes: a row's 128 are one cache line) and
// receives token p, weight rows 4 q .. 4 q + 3.  The wavefronts' sums are joined
// in shared memory in a fixed order.  Rows past the last are read as the last one and not
// stored.  1 x 8192 x 3584: 6.9 us (4.3 TB/s of weights).
#include "fp8g.h"

namespace tpmlp {
namespace g8 {

enum { F_STORE = 0, F_GLU_FWD = 1, F_GLU_BWD = 2 };
constexpr int FEW_ROWS = 64;  // of A, at most, a workgroup
constexpr int FEW_WAVES = 4;

__device__ __forceinline__ i32x8_t load_codes(const uint8_t* p) {
  const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(p);
  const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(p + 16);
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int MT, int NB, int NW, int SC, bool SQ, int FMT_A, int FMT_B, int EPI>
__global__ __launch_bounds__(64 * NW) void gemm_few(G8GemmArgs a) {
  // blocks of 16 weight rows: the gate's and the up projection's, or NB neighbours
  constexpr int MATS = EPI == F_GLU_FWD ? 2 : NB;
  static_assert(EPI != F_GLU_FWD || NB == 1);
  constexpr int U = MT <= 2 ? 4 : 2;  // groups on their way at a time
  __shared__ f32x4_t red[NW][MATS][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int p = lane & 15, q = lane >> 4;
  // (blocks of columns first: those that run together read the same rows of A)
  const int blocks_n = (a.N + 16 * NB - 1) / (16 * NB);
  const uint32_t block = a.first + blockIdx.x;
  const int n0 = (int)(block % blocks_n) * 16 * NB;
  const int64_t m_first = (int64_t)(block / blocks_n) * FEW_ROWS;
  const int64_t M = a.M;
  int n[MATS];
#pragma unroll
  for (int w = 0; w < MATS; ++w) n[w] = min(n0 + (EPI == F_GLU_FWD ? 0 : 16 * w) + p, a.N - 1);
  const int kt_part = a.K / kGroup, kt_all = kt_part * a.parts;
  const uint8_t* xrow[MT];
  int64_t m[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i] = min(m_first + 16 * i + p, M - 1);
    xrow[i] = a.A + m[i] * a.lda + 32 * q;
  }
  f32x4_t acc[MATS][MT];
#pragma unroll
  for (int w = 0; w < MATS; ++w)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[w][i] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

  for (int k0 = wave; k0 < kt_all; k0 += NW * U) {
    i32x8_t fb[U][MATS], fa[U][MT];
    float sa[U][MT], sb[U][MATS][SQ ? 1 : 4];
    int ea[U][MT], eb[U][MATS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kt = min(k0 + u * NW, kt_all - 1);
      const int part = kt >= kt_part ? 1 : 0, kb = kt - part * kt_part;
#pragma unroll
      for (int w = 0; w < MATS; ++w) {
        const bool second = EPI == F_GLU_FWD ? w == 1 : part == 1;
        fb[u][w] = load_codes((second ? a.B2 : a.B) + (int64_t)n[w] * a.K + kb * 128 + 32 * q);
        const void* s = second ? a.sB2 : a.sB;
        if constexpr (SC == TP_GROUP_F32) {
          const float* f = reinterpret_cast<const float*>(s);
          if constexpr (SQ) {
            sb[u][w][0] = f[(int64_t)(n0 / kGroup) * kt_part + kb];
          } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) sb[u][w][t] = f[(int64_t)kb * a.N + min(n0 + 16 * w + 4 * q + t, a.N - 1)];
          }
        } else {
          eb[u][w] = reinterpret_cast<const uint8_t*>(s)[SQ ? (int64_t)(n0 / kGroup) * kt_part + kb : (int64_t)kb * a.N + n[w]];
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        fa[u][i] = load_codes(xrow[i] + (int64_t)kt * 128);
        if constexpr (SC == TP_GROUP_F32) sa[u][i] = reinterpret_cast<const float*>(a.sA)[(int64_t)kt * M + m[i]];
        else ea[u][i] = reinterpret_cast<const uint8_t*>(a.sA)[(int64_t)kt * M + m[i]];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * NW >= kt_all) break;
      bf16x8g_t wb[MATS][4];
#pragma unroll
      for (int w = 0; w < MATS; ++w)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          wb[w][c] = widen<FMT_B>(fb[u][w][2 * c], fb[u][w][2 * c + 1], SC == TP_GROUP_F32 ? 1.0f : e8m0_half(eb[u][w]));
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        f32x4_t r[MATS];
#pragma unroll
        for (int w = 0; w < MATS; ++w) r[w] = SC == TP_GROUP_F32 ? (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f} : acc[w][i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bf16x8g_t wa = widen<FMT_A>(fa[u][i][2 * c], fa[u][i][2 * c + 1], SC == TP_GROUP_F32 ? 1.0f : e8m0_half(ea[u][i]));
#pragma unroll
          for (int w = 0; w < MATS; ++w) r[w] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[w][c], wa, r[w], 0, 0, 0);
        }
#pragma unroll
        for (int w = 0; w < MATS; ++w) {
          if constexpr (SC == TP_GROUP_F32) {
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[w][i][t] = fmaf(r[w][t], sa[u][i] * sb[u][w][SQ ? 0 : t], acc[w][i][t]);
          } else {
            acc[w][i] = r[w];
          }
        }
      }
    }
  }

#pragma unroll
  for (int w = 0; w < MATS; ++w)
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][w][i][lane] = acc[w][i];
  __syncthreads();
  if (wave >= MT) return;
  // wavefront i finishes tokens 16 i .. 16 i + 15
  float v[MATS][4];
#pragma unroll
  for (int w = 0; w < MATS; ++w) {
    f32x4_t s = red[0][w][wave][lane];
#pragma unroll
    for (int c = 1; c < NW; ++c) s += red[c][w][wave][lane];
#pragma unroll
    for (int t = 0; t < 4; ++t) v[w][t] = SC == TP_GROUP_E8M0 ? s[t] * E8M0_SUMS : s[t];
  }
  const int64_t row = m_first + 16 * wave + p;
  const int col = n0 + 4 * q;
  if (row >= M || col >= a.N) return;
  const int64_t off = row * a.N + col;
  const Gate gate(a.gate);
  if constexpr (EPI == F_STORE) {
#pragma unroll
    for (int w = 0; w < MATS; ++w) {
      if (col + 16 * w >= a.N) break;
      if (a.out_bf16) {
        Store4<bf16_t>::store(a.C, off + 16 * w, v[w]);
      } else {
        if (a.accumulate) {
          float c[4];
          Store4<float>::load(a.C, off + 16 * w, c);
#pragma unroll
          for (int t = 0; t < 4; ++t) v[w][t] += c[t];
        }
        Store4<float>::store(a.C, off + 16 * w, v[w]);
      }
    }
  } else if constexpr (EPI == F_GLU_FWD) {
    if (a.Z) {
      Store4<bf16_t>::store(a.Z, row * 2 * a.N + col, v[0]);
      Store4<bf16_t>::store(a.Z, row * 2 * a.N + a.N + col, v[1]);
    }
    float h[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) h[t] = gate.act(v[0][t]) * v[1][t];
    if (a.H) Store4<bf16_t>::store(a.H, off, h);
    if (a.raw) Store4<float>::store(a.raw, off, h);
  } else {
#pragma unroll
    for (int w = 0; w < MATS; ++w) {
      const int c = col + 16 * w;
      if (c >= a.N) break;
      float g[4], u[4], dg[4], du[4];
      Store4<bf16_t>::load(a.Z, row * 2 * a.N + c, g);
      Store4<bf16_t>::load(a.Z, row * 2 * a.N + a.N + c, u);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float act, slope;
        gate.both(g[t], act, slope);
        dg[t] = v[w][t] * u[t] * slope;
        du[t] = v[w][t] * act;
      }
      Store4<float>::store(a.raw, row * 2 * a.N + c, dg);
      Store4<float>::store(a.raw, row * 2 * a.N + a.N + c, du);
    }
  }
}

template <int MT, int NB, int SC, bool SQ, int FMT_A, int FMT_B, int EPI>
static hipError_t few_run(const G8GemmArgs& a, hipStream_t st) {
  const int64_t blocks = g8_over(a.N, 16 * NB) * g8_over(a.M, FEW_ROWS);
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  return g8_in_launches(blocks, [&](int64_t first, int64_t count) {
    G8GemmArgs b = a;
    b.first = (int)first;
    hipLaunchKernelGGL((gemm_few<MT, NB, FEW_WAVES, SC, SQ, FMT_A, FMT_B, EPI>), dim3((unsigned)count), dim3(64 * FEW_WAVES), 0,
                       st, b);
    return hipGetLastError();
  });
}
template <int SC, bool SQ, int FMT_A, int FMT_B, int EPI>
static hipError_t few(const G8GemmArgs& a, hipStream_t st) {
  if (a.M <= 16) return few_run<1, 1, SC, SQ, FMT_A, FMT_B, EPI>(a, st);
  if (a.M <= 32) return few_run<2, 1, SC, SQ, FMT_A, FMT_B, EPI>(a, st);
  if constexpr (EPI != F_GLU_FWD) {  // (its workgroups have 32 weight rows at any rate)
    if (g8_wide(a.M, a.N)) return few_run<4, 2, SC, SQ, FMT_A, FMT_B, EPI>(a, st);
  }
  return few_run<4, 1, SC, SQ, FMT_A, FMT_B, EPI>(a, st);
}

template <int SC, bool SQ>
static hipError_t few_formats(int fa, int fb, const G8GemmArgs& a, hipStream_t st) {
  if (fa == 0 && fb == 0) return few<SC, SQ, 0, 0, F_STORE>(a, st);
  if (fa == 1 && fb == 0) return few<SC, SQ, 1, 0, F_STORE>(a, st);
  if (fa == 0 && fb == 1) return few<SC, SQ, 0, 1, F_STORE>(a, st);
  return hipErrorInvalidValue;
}

}  // namespace g8

hipError_t g8_gemm_few_launch(int fmt_a, int fmt_b, int scale, int square, const G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (scale == TP_GROUP_F32)
    return square ? few_formats<0, true>(fmt_a, fmt_b, a, st) : few_formats<0, false>(fmt_a, fmt_b, a, st);
  return square ? few_formats<1, true>(fmt_a, fmt_b, a, st) : few_formats<1, false>(fmt_a, fmt_b, a, st);
}

hipError_t g8_glu_fwd_few_launch(int scale, const G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  return scale == TP_GROUP_F32 ? few<0, true, 0, 0, F_GLU_FWD>(a, st) : few<1, true, 0, 0, F_GLU_FWD>(a, st);
}

hipError_t g8_glu_bwd_few_launch(int fmt, int scale, const G8GemmArgs& a, hipStream_t st) {
  using namespace g8;
  if (fmt == 0)
    return scale == TP_GROUP_F32 ? few<0, true, 0, 0, F_GLU_BWD>(a, st) : few<1, true, 0, 0, F_GLU_BWD>(a, st);
  return scale == TP_GROUP_F32 ? few<0, true, 1, 0, F_GLU_BWD>(a, st) : few<1, true, 1, 0, F_GLU_BWD>(a, st);
}

}  // namespace tpmlp
