// Quantization with group scales (the formulas: include/tpmlp_fp8g.h).
//
// HBM-bound: a value is read once (2 or 4 bytes) and leaves 1 byte and 1/128
// or 4/128 of one for each orientation.  Two forms:
//  - rows: a group of 128 values is 16 lanes' (8 values a lane, one or two
//    16-byte loads), its largest magnitude a reduction within them.
//  - tile: 128 rows x 128 columns a workgroup, for squares and wherever the
//    transpose is made.  The same 16 lanes have a row; a column's largest
//    magnitude goes through the wavefront and shared memory.  Transposed codes are
//    staged as bytes and turned 4 x 4 in registers, so that a column's 128
//    codes are written by 8 neighbouring threads, 16 bytes each.
#include "fp8g.h"

namespace tpmlp {
namespace g8 {

constexpr int QNT = 256;

// 8 values of a row as fp32
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool ok, float f[8]) {
  if (ok) {
    Vec8<T>::load(p, 0, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 0.0f;
  }
}
// fp32 rows may end in the middle of 8 values
__device__ __forceinline__ void load8_part(const float* p, int n, float f[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = 0.0f;
  if (n >= 8) {
    Vec8<float>::load(p, 0, f);
  } else if (n >= 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  }
}
template <typename T>
__device__ __forceinline__ void load_row8(const T* x, int64_t off, int64_t left, float f[8]) {
  if constexpr (sizeof(T) == 4) load8_part(x + off, left > 8 ? 8 : (int)left, f);
  else load8<T>(x + off, left > 0, f);
}

__device__ __forceinline__ uint32_t top8(const float f[8]) {
  uint32_t m = mag(f[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) m = max(m, mag(f[k]));
  return m;
}

__device__ __forceinline__ uint32_t top_of_16(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = xor_max(m, d);
  return m;
}

// rows form: a workgroup takes 16 rows x QG groups a turn (the scales of the
// 16 rows lie together)
constexpr int QG = 4;
template <typename T, int FMT, int SC>
__global__ __launch_bounds__(QNT) void quant_rows(G8QuantArgs a) {
  const T* x = reinterpret_cast<const T*>(a.x);
  const int64_t groups = groups_of(a.cols), pc = groups * kGroup, ldq = pc * a.parts;
  const int64_t gb = (groups + QG - 1) / QG, rb = (a.rows + 15) / 16;
  const int64_t turns = gb * rb * a.parts;
  const int r16 = threadIdx.x >> 4, c8 = (threadIdx.x & 15) * 8;
  for (int64_t t = blockIdx.x; t < turns; t += gridDim.x) {
    const int64_t part = t / (gb * rb), u = t - part * gb * rb;
    const int64_t r = (u / gb) * 16 + r16, g0 = (u % gb) * QG;
    if (r >= a.rows) continue;  // (whole groups of 16 lanes)
    float f[QG][8];
#pragma unroll
    for (int k = 0; k < QG; ++k) {
      const int64_t c = (g0 + k) * kGroup + c8;
      load_row8<T>(x, r * a.ldx + part * a.cols + c, a.cols - c, f[k]);
    }
#pragma unroll
    for (int k = 0; k < QG; ++k) {
      const int64_t g = g0 + k;
      const GroupScale<FMT, SC> gs(top_of_16(top8(f[k])));
      if (g < groups) {
        const u32x2_t o = {codes4<FMT>(f[k][0], f[k][1], f[k][2], f[k][3], gs.inv),
                           codes4<FMT>(f[k][4], f[k][5], f[k][6], f[k][7], gs.inv)};
        *reinterpret_cast<u32x2_t*>(a.q + r * ldq + part * pc + g * kGroup + c8) = o;
        if (c8 == 0) gs.store(a.s, (part * groups + g) * a.rows + r);
      }
    }
  }
}

// tile form
constexpr int T_PITCH = 132;  // bytes of a staged row of codes
template <typename T, int FMT, int SC, bool SQ>
__global__ __launch_bounds__(QNT) void quant_tile(G8QuantArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t stage[kGroup * T_PITCH];
  __shared__ uint32_t red[QNT / 64][kGroup];
  const T* x = reinterpret_cast<const T*>(a.x);
  const int64_t gc = groups_of(a.cols), gr = groups_of(a.rows);
  const int64_t pc = gc * kGroup, pr = gr * kGroup, ldq = pc * a.parts;
  const int64_t turns = gc * gr * a.parts;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = tid >> 4, c8 = (tid & 15) * 8;
  for (int64_t t = blockIdx.x; t < turns; t += gridDim.x) {
    const int64_t part = t / (gc * gr), v = t - part * gc * gr;
    const int64_t tr = v / gc, tc = v % gc;
    const int64_t r0 = tr * kGroup, c = tc * kGroup + c8;
    float f[8][8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t r = r0 + 16 * u + r16;
      load_row8<T>(x, r * a.ldx + part * a.cols + c, r < a.rows ? a.cols - c : 0, f[u]);
    }
    float col_inv[8];
    float sq_inv = 0.0f;
    if (SQ || a.q_t) {
      // largest magnitude of each column (squares: of all)
      uint32_t m[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = mag(f[0][k]);
#pragma unroll
        for (int u = 1; u < 8; ++u) m[k] = max(m[k], mag(f[u][k]));
        m[k] = xor_max(xor_max(m[k], 16), 32);
      }
      if (lane < 16) {
#pragma unroll
        for (int k = 0; k < 8; ++k) red[wave][c8 + k] = m[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        m[k] = max(max(red[0][c8 + k], red[1][c8 + k]), max(red[2][c8 + k], red[3][c8 + k]));
      if constexpr (SQ) {
        uint32_t w = m[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) w = max(w, m[k]);
        const GroupScale<FMT, SC> gs(top_of_16(w));
        sq_inv = gs.inv;
        if (tid == 0 && a.q) gs.store(a.s, (part * gr + tr) * gc + tc);
        if (tid == 0 && a.q_t) gs.store(a.s_t, (part * gc + tc) * gr + tr);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const GroupScale<FMT, SC> gs(m[k]);
          col_inv[k] = gs.inv;
          if (tid < 16 && c + k < a.cols) gs.store(a.s_t, (part * gr + tr) * a.cols + c + k);
        }
      }
    }
    if (a.q) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t r = r0 + 16 * u + r16;
        float inv = sq_inv;
        if constexpr (!SQ) {
          const GroupScale<FMT, SC> gs(top_of_16(top8(f[u])));
          inv = gs.inv;
          if (c8 == 0 && r < a.rows) gs.store(a.s, (part * gc + tc) * a.rows + r);
        }
        if (r < a.rows) {
          const u32x2_t o = {codes4<FMT>(f[u][0], f[u][1], f[u][2], f[u][3], inv),
                             codes4<FMT>(f[u][4], f[u][5], f[u][6], f[u][7], inv)};
          *reinterpret_cast<u32x2_t*>(a.q + r * ldq + part * pc + c) = o;
        }
      }
    }
    if (a.q_t) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t* d = reinterpret_cast<uint32_t*>(stage + (16 * u + r16) * T_PITCH + c8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (SQ) {
            d[h] = codes4<FMT>(f[u][4 * h], f[u][4 * h + 1], f[u][4 * h + 2], f[u][4 * h + 3], sq_inv);
          } else {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = col_inv[4 * h + k] > 0.0f ? f[u][4 * h + k] * col_inv[4 * h + k] : 0.0f;
            d[h] = fp8x4<FMT>(y[0], y[1], y[2], y[3], 1.0f);
          }
        }
      }
      __syncthreads();
      // thread: columns 4 q .. 4 q + 3, rows 16 g .. 16 g + 15
      const int q = tid >> 3, g = tid & 7;
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = *reinterpret_cast<const uint32_t*>(stage + (16 * g + j) * T_PITCH + 4 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t col = tc * kGroup + 4 * q + i;
        if (col < a.cols) {
          u32x4_t o;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            // byte i of four words: two permutes pick pairs, one joins them
            const uint32_t lo = __builtin_amdgcn_perm(w[4 * b + 1], w[4 * b], 0x0c0c0400u + 0x0101u * i);
            const uint32_t hi = __builtin_amdgcn_perm(w[4 * b + 3], w[4 * b + 2], 0x0c0c0400u + 0x0101u * i);
            o[b] = lo | (hi << 16);
          }
          *reinterpret_cast<u32x4_t*>(a.q_t + (part * a.cols + col) * pr + r0 + 16 * g) = o;
        }
      }
      __syncthreads();  // the stage and the sums are rewritten by the next turn
    } else if constexpr (SQ) {
      __syncthreads();
    }
  }
}

template <typename T, int FMT, int SC>
static hipError_t quant_run(int square, const G8QuantArgs& a, hipStream_t st) {
  const bool tile = square || a.q_t;
  const int64_t turns = (tile ? groups_of(a.cols) * groups_of(a.rows)
                              : (groups_of(a.cols) + QG - 1) / QG * ((a.rows + 15) / 16)) * a.parts;
  const dim3 grid((unsigned)(turns < (1 << 20) ? turns : (1 << 20)));
  if (!tile)
    hipLaunchKernelGGL((quant_rows<T, FMT, SC>), grid, dim3(QNT), 0, st, a);
  else if (square)
    hipLaunchKernelGGL((quant_tile<T, FMT, SC, true>), grid, dim3(QNT), 0, st, a);
  else
    hipLaunchKernelGGL((quant_tile<T, FMT, SC, false>), grid, dim3(QNT), 0, st, a);
  return hipGetLastError();
}

}  // namespace g8

hipError_t g8_quant_launch(int dtype, int fmt, int scale, int square, const G8QuantArgs& a, hipStream_t st) {
  if (a.rows == 0 || (!a.q && !a.q_t)) return hipSuccess;
  using namespace g8;
#define RUN(T, F, S) return quant_run<T, F, S>(square, a, st)
  if (dtype == TP_BF16) {
    if (fmt == 0) { if (scale == TP_GROUP_F32) RUN(bf16_t, 0, 0); RUN(bf16_t, 0, 1); }
    if (scale == TP_GROUP_F32) RUN(bf16_t, 1, 0);
    RUN(bf16_t, 1, 1);
  }
  if (fmt == 0) { if (scale == TP_GROUP_F32) RUN(float, 0, 0); RUN(float, 0, 1); }
  if (scale == TP_GROUP_F32) RUN(float, 1, 0);
  RUN(float, 1, 1);
#undef RUN
}

}  // namespace tpmlp
