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
//    codes are written by 8 neighbouring threads, 16 bytes each.  4096 x 8192 bf16 both
//    ways 29.4 us (4.6 TB/s), 8192 x 3584 fp32 in squares both ways 36 (4.9).
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

// tile form.  A lane's 8 neighbouring values of a row, as loaded: bf16 ones
// are compared two at a time, as 15-bit magnitudes.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
template <typename T> struct Eight;
template <> struct Eight<bf16_t> {
  static constexpr int W = 4;  // words of magnitudes
  uint32_t w[4];
  __device__ __forceinline__ void load(const bf16_t* x, int64_t off, int64_t left) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (left > 0) v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(x + off));
    *reinterpret_cast<u32x4_t*>(w) = v;
  }
  __device__ __forceinline__ float value(int k) const {
    return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  }
  __device__ __forceinline__ uint32_t mags(int i) const { return w[i] & 0x7fff7fffu; }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) { return max_u16x2(a, b); }
  // fp32 magnitude of a word's value, and of the larger of its two
  static __device__ __forceinline__ uint32_t one(const uint32_t* m, int k) { return k & 1 ? m[k / 2] & 0xffff0000u : m[k / 2] << 16; }
  static __device__ __forceinline__ uint32_t whole(uint32_t m) { return max(m & 0xffff0000u, m << 16); }
};
template <> struct Eight<float> {
  static constexpr int W = 8;
  float f[8];
  __device__ __forceinline__ void load(const float* x, int64_t off, int64_t left) { load8_part(x + off, left > 8 ? 8 : (int)left, f); }
  __device__ __forceinline__ float value(int k) const { return f[k]; }
  __device__ __forceinline__ uint32_t mags(int i) const { return mag(f[i]); }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t one(const uint32_t* m, int k) { return m[k]; }
  static __device__ __forceinline__ uint32_t whole(uint32_t m) { return m; }
};

constexpr int T_PITCH = 132;  // bytes of a staged row of codes
template <typename T, int FMT, int SC, bool SQ>
__global__ __launch_bounds__(QNT, 4) void quant_tile(G8QuantArgs a) {
  typedef Eight<T> E;
  __shared__ __attribute__((aligned(16))) uint8_t stage[kGroup * T_PITCH];
  __shared__ uint32_t red[QNT / 64][16 * E::W];
  __shared__ float inverse[kGroup];
  const T* x = reinterpret_cast<const T*>(a.x);
  const int64_t gc = groups_of(a.cols), gr = groups_of(a.rows);
  const int64_t pc = gc * kGroup, pr = gr * kGroup, ldq = pc * a.parts;
  const int64_t turns = gc * gr * a.parts;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = tid >> 4, l16 = tid & 15, c8 = l16 * 8;
  for (int64_t t = blockIdx.x; t < turns; t += gridDim.x) {
    const int64_t part = t / (gc * gr), v = t - part * gc * gr;
    const int64_t tr = v / gc, tc = v % gc;
    const int64_t r0 = tr * kGroup, c = tc * kGroup + c8;
    E e[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t r = r0 + 16 * u + r16;
      e[u].load(x, r * a.ldx + part * a.cols + c, r < a.rows ? a.cols - c : 0);
    }
    float sq_inv = 0.0f;
    if (SQ || a.q_t) {
      // largest magnitude of each column over the rows of a thread, a
      // wavefront, the workgroup
#pragma unroll
      for (int i = 0; i < E::W; ++i) {
        uint32_t m = e[0].mags(i);
#pragma unroll
        for (int u = 1; u < 8; ++u) m = E::most(m, e[u].mags(i));
        m = E::most(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = E::most(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (lane < 16) red[wave][l16 * E::W + i] = m;
      }
      __syncthreads();
      if constexpr (SQ) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < E::W; ++i) {
          const int at = l16 * E::W + i;
          w = E::most(w, E::most(E::most(red[0][at], red[1][at]), E::most(red[2][at], red[3][at])));
        }
        const GroupScale<FMT, SC> gs(top_of_16(E::whole(w)));
        sq_inv = gs.inv;
        if (tid == 0 && a.q) gs.store(a.s, (part * gr + tr) * gc + tc);
        if (tid == 0 && a.q_t) gs.store(a.s_t, (part * gc + tc) * gr + tr);
      } else {
        if (tid < kGroup) {  // a column each
          uint32_t m[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = E::one(red[k] + tid / 8 * E::W, tid % 8);
          const GroupScale<FMT, SC> gs(max(max(m[0], m[1]), max(m[2], m[3])));
          inverse[tid] = gs.inv;
          if (tc * kGroup + tid < a.cols) gs.store(a.s_t, (part * gr + tr) * a.cols + tc * kGroup + tid);
        }
        __syncthreads();
      }
    }
    if (a.q) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t r = r0 + 16 * u + r16;
        float inv = sq_inv;
        if constexpr (!SQ) {
          uint32_t m = e[u].mags(0);
#pragma unroll
          for (int i = 1; i < E::W; ++i) m = E::most(m, e[u].mags(i));
          const GroupScale<FMT, SC> gs(top_of_16(E::whole(m)));
          inv = gs.inv;
          if (l16 == 0 && r < a.rows) gs.store(a.s, (part * gc + tc) * a.rows + r);
        }
        if (r < a.rows) {
          const u32x2_t o = {codes4<FMT>(e[u].value(0), e[u].value(1), e[u].value(2), e[u].value(3), inv),
                             codes4<FMT>(e[u].value(4), e[u].value(5), e[u].value(6), e[u].value(7), inv)};
          *reinterpret_cast<u32x2_t*>(a.q + r * ldq + part * pc + c) = o;
        }
      }
    }
    if (a.q_t) {
      float ci[8];
      bool plain = true;  // (a column without a scale: zeros, whatever it holds)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ci[k] = SQ ? sq_inv : inverse[c8 + k];
        plain = plain && ci[k] > 0.0f;
      }
      plain = __all(plain);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        uint32_t* d = reinterpret_cast<uint32_t*>(stage + (16 * u + r16) * T_PITCH + c8);
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = e[u].value(k) * ci[k];
        if (!plain) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = ci[k] > 0.0f ? y[k] : 0.0f;
        }
        d[0] = pack4<FMT>(y[0], y[1], y[2], y[3]);
        d[1] = pack4<FMT>(y[4], y[5], y[6], y[7]);
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
    }
    __syncthreads();  // the stage and the sums are rewritten by the next turn
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
