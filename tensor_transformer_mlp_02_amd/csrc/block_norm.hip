// The seam between two blocks: norm after a block, gate and residual scale,
// residual sum and the next block's norm, forward and backward
// (Megatron Core 带读 §03: norm -> block -> residual, layer by layer).
//
// Per token, with xh = (t - mu) r of either norm:
//   u = oh w_post + b_post,  y = a x + b gate u,  h = yh w_pre + b_pre
// backward, p = dh w_pre, D = dY + r_y (p - mean p - yh mean(p yh)):
//   dX = a D,  dgate = b sum D u,  du = b gate D,
//   q = du w_post,  dO = r_o (q - mean q - oh mean(q oh))
// (the plain means only for the LayerNorm), and the column sums
//   dw_pre = sum dh yh, db_pre = sum dh, dw_post = sum du oh, db_post = sum du.
// Both directions move whole rows and are HBM-bound.
#include "block_launch.h"
#include "common.h"

namespace tpmlp {
namespace norm {

constexpr int NT = 256;
// Threads in flight for each of the 256 compute units where workgroups walk
// over rows: 512 (8 wavefronts with the next row requested ahead).  Forward,
// 4096 x 8192 bf16: 53 us at 512 threads, 55 at 1024, 57 at 2048, 74 with a
// workgroup for each row; 1500 x 5120: 16.2, 17.5, 19.9 us.
constexpr int CU_THREADS = 512, CUS = 256;

// one 16-byte piece of a row as floats
template <typename T> struct Piece;
template <> struct Piece<bf16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float v[8]) {
    Vec8<bf16_t>::load(p, i, v);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float v[8]) {
    Vec8<bf16_t>::store(p, i, v);
  }
};
template <> struct Piece<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void load(const void* p, int64_t i, float v[4]) {
    Store4<float>::load(p, i, v);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float v[4]) {
    Store4<float>::store(p, i, v);
  }
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}

// sum over the workgroup, the same in every thread (fixed order)
__device__ __forceinline__ float block_sum(float x, float* red) {
  x = wave_sum(x);
  __syncthreads();  // red may still be read from the sum before
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) t += red[w];
  return t;
}

// ---------------------------------------------------------------------------
// Rows that stay in registers: TPR threads share a row, P 16-byte pieces
// each, so that every tensor is read from memory once.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 load_raw(const void* p, int64_t piece) {
  return reinterpret_cast<const uint4*>(p)[piece];
}
template <typename T>
__device__ __forceinline__ void store_piece(void* p, int64_t piece, const float v[Piece<T>::V]) {
  Piece<T>::store(p, piece * Piece<T>::V, v);
}
template <typename T>
__device__ __forceinline__ void unpack(const uint4& r, float v[Piece<T>::V]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (Piece<T>::V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  }
}

// sum over a wavefront, in every lane: data-parallel moves within rows of
// 16 lanes and across them, without a trip through shared memory
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, true);
  return x + __int_as_float(y);
}
__device__ __forceinline__ float wave_total(float x) {
  x = dpp_add<0x111, 0xf>(x);  // row_shr:1, 2, 4, 8
  x = dpp_add<0x112, 0xf>(x);
  x = dpp_add<0x114, 0xf>(x);
  x = dpp_add<0x118, 0xf>(x);
  x = dpp_add<0x142, 0xa>(x);  // row_bcast:15 into rows 1 and 3
  x = dpp_add<0x143, 0xc>(x);  // row_bcast:31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// the same over each 8, 16 or 32 lanes
template <int LANES>
__device__ __forceinline__ float lanes_total(float x) {
  x = dpp_add<0xB1, 0xf>(x);   // lane ^ 1
  x = dpp_add<0x4E, 0xf>(x);   // lane ^ 2
  x = dpp_add<0x141, 0xf>(x);  // within 8: lane 7 - i
  if constexpr (LANES >= 16) x = dpp_add<0x140, 0xf>(x);  // within 16: lane 15 - i
  if constexpr (LANES == 32) {
    const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(v[0]) + __uint_as_float(v[1]);
  }
  return x;
}

template <int TPR>
struct Rows {
  static constexpr int THREADS = TPR < 256 ? 256 : TPR;
  static constexpr int AT_ONCE = THREADS / TPR;  // rows of a workgroup
};

// K sums over the threads of each row.  `red` has two halves used in turn:
// one barrier a call, since a wavefront that writes a half again has passed
// the barrier behind every read of it.
template <int TPR, int K, int THREADS = Rows<TPR>::THREADS>
__device__ __forceinline__ void row_sums(float (&v)[K], float* red, int& half) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (TPR < 64) v[k] = lanes_total<TPR>(v[k]);
    else v[k] = wave_total(v[k]);
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    float* mine = red + half * (THREADS / 64) * K;
    half ^= 1;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) mine[wave * K + k] = v[k];
    __syncthreads();
    const float* row = mine + (wave / W) * W * K;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = row[k];
#pragma unroll
      for (int w = 1; w < W; ++w) t += row[w * K + k];
      v[k] = t;
    }
  }
}

// the compiler forgets what it knows of v: values unpacked from it do not
// stay in registers past here
__device__ __forceinline__ void hold(uint4& v) {
  asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w));
}

// The weights are kept in registers over a workgroup's rows, and the next
// row is requested before the present one is summed.  HBM-bound: 4096 x 8192
// bf16 with both norms and a gate 53 us, 5.1 TB/s, the rate of a large copy;
// non-temporal loads or stores change nothing.
template <typename T, bool LAYER, int TPR, int P>
__global__ __launch_bounds__(Rows<TPR>::THREADS) void fwd_kernel(NormFwdArgs A) {
  constexpr int V = Piece<T>::V, R = Rows<TPR>::AT_ONCE;
  __shared__ float red[2 * (Rows<TPR>::THREADS / 64)];
  int half = 0;
  const int tr = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const int pieces = A.H / V;
  const float inv_h = 1.0f / (float)A.H;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  bool in[P];
  uint4 w_post[P], b_post[P], gate[P], w_pre[P], b_pre[P], x[P], o[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int c = tr + p * TPR;
    in[p] = c < pieces;
    w_post[p] = A.w_post && in[p] ? load_raw(A.w_post, c) : zero;
    b_post[p] = A.b_post && in[p] ? load_raw(A.b_post, c) : zero;
    gate[p] = A.G == 1 && in[p] ? load_raw(A.gate, c) : zero;
    w_pre[p] = A.w_pre && in[p] ? load_raw(A.w_pre, c) : zero;
    b_pre[p] = A.b_pre && in[p] ? load_raw(A.b_pre, c) : zero;
    x[p] = o[p] = zero;
  }
  const int64_t stride = (int64_t)gridDim.x * R;
  auto request = [&](int64_t n, uint4 (&xx)[P], uint4 (&oo)[P]) {
    if (n >= A.N) return;
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (in[p]) {
        xx[p] = load_raw(A.X, n * pieces + tr + p * TPR);
        if (A.O) oo[p] = load_raw(A.O, n * pieces + tr + p * TPR);
      }
  };
  const int64_t first = (int64_t)blockIdx.x * R;
  request(first + rg, x, o);
  for (int64_t base = first; base < A.N; base += stride) {
    const int64_t n = base + rg;
    const bool live = n < A.N;
    uint4 xn[P], on[P], gt[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      xn[p] = on[p] = zero;
      gt[p] = gate[p];
    }
    if (A.G > 1 && live) {
      const int64_t g = (int64_t)((uint32_t)n % (uint32_t)A.G) * pieces;
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (in[p]) gt[p] = load_raw(A.gate, g + tr + p * TPR);
    }
    // the next row is asked for at once; where four bf16 pieces fill the
    // registers, when this row's are free, and its values are unpacked again
    // after the sums (2048 x 16384: 46 us so, 50 otherwise, with biases and
    // means 56 and 169)
    constexpr bool AHEAD = V * P < 32;
    if constexpr (AHEAD) request(n + stride, xn, on);
    float mo = 0.f, ro = 1.f;
    if (A.w_post) {
      if constexpr (LAYER) {
        float s[1] = {0.f};
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float t[V];
          unpack<T>(o[p], t);
#pragma unroll
          for (int i = 0; i < V; ++i) s[0] += t[i];
        }
        row_sums<TPR>(s, red, half);
        mo = s[0] * inv_h;
      }
      float s[1] = {0.f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float t[V];
        unpack<T>(o[p], t);
#pragma unroll
        for (int i = 0; i < V; ++i) s[0] += in[p] || !LAYER ? (t[i] - mo) * (t[i] - mo) : 0.f;
      }
      row_sums<TPR>(s, red, half);
      ro = 1.0f / sqrtf(s[0] * inv_h + A.eps);
      if (A.stat_post && tr == 0 && live) {
        A.stat_post[n] = ro;
        if constexpr (LAYER) A.stat_post[A.N + n] = mo;
      }
    }
    if constexpr (!AHEAD) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        hold(o[p]);
        hold(x[p]);
      }
    }
    float y[P][V];
    float sy[1] = {0.f}, sq[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      unpack<T>(x[p], y[p]);
      if (A.O) {
        float u[V], w[V];
        unpack<T>(o[p], u);
        if (A.w_post) {
          unpack<T>(w_post[p], w);
#pragma unroll
          for (int i = 0; i < V; ++i) u[i] = (u[i] - mo) * ro * w[i];
          if (A.b_post) {
            unpack<T>(b_post[p], w);
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] += w[i];
          }
        }
        if (A.G > 0) {
          unpack<T>(gt[p], w);
#pragma unroll
          for (int i = 0; i < V; ++i) u[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) y[p][i] = A.a * y[p][i] + A.b * u[i];
        if (in[p] && live) store_piece<T>(A.Y, n * pieces + tr + p * TPR, y[p]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        sy[0] += y[p][i];
        sq[0] += y[p][i] * y[p][i];
      }
    }
    if constexpr (!AHEAD) request(n + stride, x, o);
    if (A.w_pre) {
      float my = 0.f;
      if constexpr (LAYER) {
        row_sums<TPR>(sy, red, half);
        my = sy[0] * inv_h;
        sq[0] = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i) sq[0] += in[p] ? (y[p][i] - my) * (y[p][i] - my) : 0.f;
      }
      row_sums<TPR>(sq, red, half);
      const float ry = 1.0f / sqrtf(sq[0] * inv_h + A.eps);
      if (A.stat_pre && tr == 0 && live) {
        A.stat_pre[n] = ry;
        if constexpr (LAYER) A.stat_pre[A.N + n] = my;
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float w[V];
        unpack<T>(w_pre[p], w);
#pragma unroll
        for (int i = 0; i < V; ++i) y[p][i] = (y[p][i] - my) * ry * w[i];
        if (A.b_pre) {
          unpack<T>(b_pre[p], w);
#pragma unroll
          for (int i = 0; i < V; ++i) y[p][i] += w[i];
        }
        if (in[p] && live) store_piece<T>(A.Hn, n * pieces + tr + p * TPR, y[p]);
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        x[p] = xn[p];
        o[p] = on[p];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Rows of any width: one workgroup walks a row in several passes
// ---------------------------------------------------------------------------
template <typename T, bool LAYER>
__global__ __launch_bounds__(NT) void fwd_wide_kernel(NormFwdArgs A) {
  constexpr int V = Piece<T>::V;
  __shared__ float red[NT / 64];
  const float inv_h = 1.0f / (float)A.H;
  for (int64_t n = blockIdx.x; n < A.N; n += gridDim.x) {
    const int64_t row = n * A.H;
    const int64_t grow = A.G > 0 ? (n % A.G) * A.H : 0;
    float mo = 0.f, ro = 1.f;
    if (A.w_post) {
      if constexpr (LAYER) {
        float s = 0.f;
        for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
          float o[V];
          Piece<T>::load(A.O, row + c, o);
#pragma unroll
          for (int i = 0; i < V; ++i) s += o[i];
        }
        mo = block_sum(s, red) * inv_h;
      }
      float s = 0.f;
      for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
        float o[V];
        Piece<T>::load(A.O, row + c, o);
#pragma unroll
        for (int i = 0; i < V; ++i) s += (o[i] - mo) * (o[i] - mo);
      }
      ro = 1.0f / sqrtf(block_sum(s, red) * inv_h + A.eps);
      if (A.stat_post && threadIdx.x == 0) {
        A.stat_post[n] = ro;
        if constexpr (LAYER) A.stat_post[A.N + n] = mo;
      }
    }
    auto y_at = [&](int c, float y[V]) {
      Piece<T>::load(A.X, row + c, y);
      if (!A.O) return;
      float u[V];
      Piece<T>::load(A.O, row + c, u);
      if (A.w_post) {
        float w[V];
        Piece<T>::load(A.w_post, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = (u[i] - mo) * ro * w[i];
        if (A.b_post) {
          Piece<T>::load(A.b_post, c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) u[i] += w[i];
        }
      }
      if (A.G > 0) {
        float g[V];
        Piece<T>::load(A.gate, grow + c, g);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = A.a * y[i] + A.b * u[i];
    };
    float my = 0.f, ry = 0.f;
    if (A.w_pre) {
      if constexpr (LAYER) {
        float s = 0.f;
        for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
          float y[V];
          y_at(c, y);
#pragma unroll
          for (int i = 0; i < V; ++i) s += y[i];
        }
        my = block_sum(s, red) * inv_h;
      }
      float s = 0.f;
      for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
        float y[V];
        y_at(c, y);
#pragma unroll
        for (int i = 0; i < V; ++i) s += (y[i] - my) * (y[i] - my);
      }
      ry = 1.0f / sqrtf(block_sum(s, red) * inv_h + A.eps);
      if (A.stat_pre && threadIdx.x == 0) {
        A.stat_pre[n] = ry;
        if constexpr (LAYER) A.stat_pre[A.N + n] = my;
      }
    }
    // Y may be X: a thread's own pieces are read for the last time before
    // they are written
    for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
      float y[V], w[V];
      y_at(c, y);
      if (A.O) Piece<T>::store(A.Y, row + c, y);
      if (A.w_pre) {
        Piece<T>::load(A.w_pre, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = (y[i] - my) * ry * w[i];
        if (A.b_pre) {
          Piece<T>::load(A.b_pre, c, w);
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] += w[i];
        }
        Piece<T>::store(A.Hn, row + c, y);
      }
    }
  }
}

// D of one piece: dY + r_y (p - m2 - yh m1), m1 = mean(p yh), m2 = mean p
template <typename T, bool LAYER>
__device__ __forceinline__ void d_at(const NormBwdArgs& A, int64_t row, int c, float ry, float my,
                                     float m1, float m2, float D[Piece<T>::V]) {
  constexpr int V = Piece<T>::V;
  if (A.dY) {
    Piece<T>::load(A.dY, row + c, D);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) D[i] = 0.f;
  }
  if (A.w_pre) {
    float g[V], w[V], y[V];
    Piece<T>::load(A.dH, row + c, g);
    Piece<T>::load(A.w_pre, c, w);
    Piece<T>::load(A.Y, row + c, y);
#pragma unroll
    for (int i = 0; i < V; ++i) D[i] += ry * (g[i] * w[i] - m2 - (y[i] - my) * ry * m1);
  }
}

// Rows of any width, row part: dX, dO, and each row's two means (ws)
template <typename T, bool LAYER>
__global__ __launch_bounds__(NT) void bwd_wide_rows_kernel(NormBwdArgs A, float* means) {
  constexpr int V = Piece<T>::V;
  __shared__ float red[NT / 64];
  const float inv_h = 1.0f / (float)A.H;
  for (int64_t n = blockIdx.x; n < A.N; n += gridDim.x) {
    const int64_t row = n * A.H;
    const int64_t grow = A.G > 0 ? (n % A.G) * A.H : 0;
    float ry = 0.f, my = 0.f, m1 = 0.f, m2 = 0.f;
    if (A.w_pre) {
      ry = A.stat_pre[n];
      if constexpr (LAYER) my = A.stat_pre[A.N + n];
      float s1 = 0.f, s2 = 0.f;
      for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
        float g[V], w[V], y[V];
        Piece<T>::load(A.dH, row + c, g);
        Piece<T>::load(A.w_pre, c, w);
        Piece<T>::load(A.Y, row + c, y);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s1 += g[i] * w[i] * ((y[i] - my) * ry);
          s2 += g[i] * w[i];
        }
      }
      m1 = block_sum(s1, red) * inv_h;
      if constexpr (LAYER) m2 = block_sum(s2, red) * inv_h;
    }
    if (threadIdx.x == 0) {
      means[2 * n] = m1;
      means[2 * n + 1] = m2;
    }
    auto q_at = [&](int c, const float D[V], float q[V]) {
#pragma unroll
      for (int i = 0; i < V; ++i) q[i] = A.b * D[i];
      if (A.G > 0) {
        float g[V];
        Piece<T>::load(A.gate, grow + c, g);
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] *= g[i];
      }
      if (A.w_post) {
        float w[V];
        Piece<T>::load(A.w_post, c, w);
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] *= w[i];
      }
    };
    float ro = 1.f, mo = 0.f, t1 = 0.f, t2 = 0.f;
    if (A.w_post) {
      ro = A.stat_post[n];
      if constexpr (LAYER) mo = A.stat_post[A.N + n];
      float s1 = 0.f, s2 = 0.f;
      for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
        float D[V], q[V], o[V];
        d_at<T, LAYER>(A, row, c, ry, my, m1, m2, D);
        q_at(c, D, q);
        Piece<T>::load(A.O, row + c, o);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s1 += q[i] * ((o[i] - mo) * ro);
          s2 += q[i];
        }
      }
      t1 = block_sum(s1, red) * inv_h;
      if constexpr (LAYER) t2 = block_sum(s2, red) * inv_h;
    }
    for (int c = threadIdx.x * V; c < A.H; c += NT * V) {
      float D[V], x[V];
      d_at<T, LAYER>(A, row, c, ry, my, m1, m2, D);
      if (A.O) {
        float q[V], o[V];
        q_at(c, D, q);
        if (A.w_post) {
          Piece<T>::load(A.O, row + c, o);
#pragma unroll
          for (int i = 0; i < V; ++i) q[i] = ro * (q[i] - t2 - (o[i] - mo) * ro * t1);
        }
        Piece<T>::store(A.dO, row + c, q);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = A.O ? A.a * D[i] : D[i];
      Piece<T>::store(A.dX, row + c, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Column sums.  The rows are dealt to W workers by their gate row, so that
// a worker holds the sums of one gate row at a time:
//   G <= W: worker w takes gate row w % G and every (W/G)-th of its tokens,
//           starting at w / G (W is a multiple of G)
//   G > W:  worker w takes the gate rows w, w + W, ... with all their
//           tokens; it finishes each gate row's gradient by itself and
//           keeps b gate A1, b gate A0 summed over its gate rows
// The partial sums [4][W][H] are added over w, in order, by reduce_kernel.
// ---------------------------------------------------------------------------
enum { SUM_W_PRE = 0, SUM_B_PRE = 1, SUM_1 = 2, SUM_0 = 3, SUMS = 4 };

template <typename T, bool LAYER>
__global__ __launch_bounds__(NT) void bwd_wide_columns_kernel(NormBwdArgs A, const float* means) {
  constexpr int V = Piece<T>::V;
  const int c = (blockIdx.x * NT + threadIdx.x) * V;
  if (c >= A.H) return;
  const int w = blockIdx.y, W = A.workers;
  const int64_t G = A.G > 0 ? A.G : 1;
  const bool many = G > W;
  float acc[SUMS][V], s_1[V], s_0[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s_1[i] = s_0[i] = 0.f;
#pragma unroll
    for (int k = 0; k < SUMS; ++k) acc[k][i] = 0.f;
  }
  auto add_row = [&](int64_t n) {
    const int64_t row = n * A.H;
    float ry = 0.f, my = 0.f, ro = 1.f, mo = 0.f, D[V];
    if (A.w_pre) {
      ry = A.stat_pre[n];
      if constexpr (LAYER) my = A.stat_pre[A.N + n];
      float g[V], y[V];
      Piece<T>::load(A.dH, row + c, g);
      Piece<T>::load(A.Y, row + c, y);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[SUM_W_PRE][i] += g[i] * ((y[i] - my) * ry);
        acc[SUM_B_PRE][i] += g[i];
      }
    }
    if (!A.O) return;
    d_at<T, LAYER>(A, row, c, ry, my, means[2 * n], means[2 * n + 1], D);
    float o[V];
    Piece<T>::load(A.O, row + c, o);
    if (A.w_post) {
      ro = A.stat_post[n];
      if constexpr (LAYER) mo = A.stat_post[A.N + n];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[SUM_1][i] += D[i] * ((o[i] - mo) * ro);
      acc[SUM_0][i] += D[i];
    }
  };
  if (!many) {
    for (int64_t n = w % G + (w / G) * G; n < A.N; n += (int64_t)W / G * G) add_row(n);
  } else {
    float wp[V], bp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) { wp[i] = 1.f; bp[i] = 0.f; }
    if (A.w_post) Piece<T>::load(A.w_post, c, wp);
    if (A.b_post) Piece<T>::load(A.b_post, c, bp);
    for (int64_t g = w; g < G; g += W) {
      for (int64_t n = g; n < A.N; n += G) add_row(n);
      float q[V];
      Piece<T>::load(A.gate, g * A.H + c, q);
      float* out = A.dgate + g * A.H + c;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = A.b * (wp[i] * acc[SUM_1][i] + bp[i] * acc[SUM_0][i]);
        out[i] = d + (A.accumulate ? out[i] : 0.f);
        s_1[i] += A.b * q[i] * acc[SUM_1][i];
        s_0[i] += A.b * q[i] * acc[SUM_0][i];
        acc[SUM_1][i] = acc[SUM_0][i] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[SUM_1][i] = s_1[i];
      acc[SUM_0][i] = s_0[i];
    }
  }
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
    float* out = A.ws + ((int64_t)k * W + w) * A.H + c;
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = acc[k][i];
  }
}

// ---------------------------------------------------------------------------
// Backward with rows in registers.  Every tensor is read once, all of a
// row's sums come from one pass: with k = b gate w_post,
//   S1 = sum p yh, S2 = sum p, and since q = k D is linear in S1 and S2,
//   sum q oh = sum k oh (dY + r p) - r (S2/H sum k oh + S1/H sum k oh yh),
//   sum q likewise without oh.
// Column sums stay in the thread that owns the columns.  The post norm's
// need only A1 = sum D oh and A0 = sum D of one gate row at a time:
//   dw_post = b sum_g gate_g A1_g,  dgate_g = b (w_post A1_g + b_post A0_g).
// ---------------------------------------------------------------------------
template <int TPR>
struct BwdRows {
  static constexpr int THREADS = TPR > CU_THREADS ? TPR : CU_THREADS;
  static constexpr int AT_ONCE = THREADS / TPR;
};

// AGAIN: after the row sums the values are unpacked from their pieces again,
// so that they do not stay in registers meanwhile (see again_pays).
template <typename T, bool LAYER, bool BIAS, bool MANY, bool AGAIN, int TPR, int P>
__global__ __launch_bounds__(BwdRows<TPR>::THREADS) void bwd_kernel(NormBwdArgs A) {
  constexpr int V = Piece<T>::V, R = BwdRows<TPR>::AT_ONCE, THREADS = BwdRows<TPR>::THREADS;
  constexpr int SUMS_ROW = LAYER ? 8 : 3;
  extern __shared__ float lds[];
  int half = 0;
  const int tr = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const int pieces = A.H / V;
  const float inv_h = 1.0f / (float)A.H;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int w = blockIdx.x, W = A.workers;
  const uint32_t G = A.G > 0 ? (uint32_t)A.G : 1u;

  bool in[P];
  uint4 w_post[P], w_pre[P], gate[P];
  uint4 dy[P], dh[P], yy[P], oo[P];
  // 16 wavefronts leave 128 registers a lane: there the two sums that every
  // call may ask for are kept in shared memory, each thread's own.  (bf16 rows
  // still spill 18 registers with a LayerNorm and 27 with an RMS norm.)
  constexpr bool KEPT = TPR > CU_THREADS && !MANY && !BIAS;
  __shared__ float kept[KEPT ? 2 * P * V * THREADS : 1];
  float a_wpre[KEPT ? 1 : P][V], a_1[KEPT ? 1 : P][V], a_bpre[BIAS ? P : 1][V], a_0[BIAS ? P : 1][V];
  // gate-weighted, of the gate rows done
  float s_1[MANY ? P : 1][V], s_0[MANY && BIAS ? P : 1][V];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    in[p] = tr + p * TPR < pieces;
    w_post[p] = A.w_post && in[p] ? load_raw(A.w_post, tr + p * TPR) : zero;
    w_pre[p] = A.w_pre && in[p] ? load_raw(A.w_pre, tr + p * TPR) : zero;
    gate[p] = dy[p] = dh[p] = yy[p] = oo[p] = zero;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (KEPT) {
        kept[(p * V + i) * THREADS + tr] = kept[((P + p) * V + i) * THREADS + tr] = 0.f;
      } else {
        a_wpre[p][i] = a_1[p][i] = 0.f;
      }
      if constexpr (BIAS) a_bpre[p][i] = a_0[p][i] = 0.f;
      if constexpr (MANY) s_1[p][i] = 0.f;
      if constexpr (MANY && BIAS) s_0[p][i] = 0.f;
    }
  }
  // this row group's rows, turn by turn; all groups of a workgroup take the
  // same number of turns, some without a row
  const uint32_t N = (uint32_t)A.N;
  uint32_t turns, per_gate = 1, g_first, g_step = 0, n_first = 0, n_step = 0;
  if constexpr (!MANY) {
    const uint32_t slices = (uint32_t)W / G;
    g_first = (uint32_t)w % G;
    const uint32_t n0 = g_first + ((uint32_t)w / G) * G;
    n_first = n0 + slices * rg * G;
    n_step = slices * R * G;
    turns = n0 < N ? (N - n0 + n_step - 1) / n_step : 0;
  } else {
    per_gate = (N + G - 1) / G;
    g_first = (uint32_t)w * R + rg;
    g_step = (uint32_t)W * R;
    turns = (G + g_step - 1) / g_step * per_gate;
  }
  auto gate_of = [&](uint32_t it) { return g_first + it / per_gate * g_step; };
  auto row_of = [&](uint32_t it) -> uint32_t {  // N: none
    if constexpr (!MANY) return min(n_first + it * n_step, N);
    const uint32_t g = gate_of(it);
    return g < G ? min(g + it % per_gate * G, N) : N;
  };
  auto load_gate = [&](uint32_t g) {
    if (A.G > 0 && g < G)
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (in[p]) gate[p] = load_raw(A.gate, (int64_t)g * pieces + tr + p * TPR);
  };
  auto request = [&](uint32_t n, uint4 (&y0)[P], uint4 (&h0)[P], uint4 (&yr)[P], uint4 (&o0)[P],
                     float (&st)[4]) {
#pragma unroll
    for (int p = 0; p < P; ++p) y0[p] = h0[p] = yr[p] = o0[p] = zero;
    st[0] = st[1] = st[2] = st[3] = 0.f;
    if (n >= N) return;
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (in[p]) {
        const int64_t at = (int64_t)n * pieces + tr + p * TPR;
        if (A.dY) y0[p] = load_raw(A.dY, at);
        if (A.w_pre) {
          h0[p] = load_raw(A.dH, at);
          yr[p] = load_raw(A.Y, at);
        }
        if (A.O) o0[p] = load_raw(A.O, at);
      }
    if (A.w_pre) {
      st[0] = A.stat_pre[n];
      if constexpr (LAYER) st[1] = A.stat_pre[A.N + n];
    }
    st[2] = 1.f;
    if (A.w_post) {
      st[2] = A.stat_post[n];
      if constexpr (LAYER) st[3] = A.stat_post[A.N + n];
    }
  };
  float st[4];
  request(turns > 0 ? row_of(0) : N, dy, dh, yy, oo, st);
  // one gate row for all of a worker's tokens: b gate w_post (b gate without a
  // norm), once (8192 x 4096 with biases 102 us without, 88 so)
  float kw[MANY ? 1 : P][V];
  if constexpr (!MANY) {
    load_gate(g_first);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float q[V], t[V];
      unpack<T>(gate[p], q);
      unpack<T>(w_post[p], t);
#pragma unroll
      for (int i = 0; i < V; ++i)
        kw[p][i] = A.b * (A.G > 0 ? q[i] : 1.f) * (A.w_post ? t[i] : in[p] ? 1.f : 0.f);
    }
  }

  for (uint32_t it = 0; it < turns; ++it) {
    const uint32_t n = row_of(it);
    const bool live = n < N;
    if (MANY && it % per_gate == 0) load_gate(gate_of(it));
    // the next row's loads on their way, where registers are left for it.  The
    // sums of many gate rows leave too few beside two bf16 pieces: 8192 x 4096
    // with a gate a token 132 us so, 124 without, with biases 252 and 168; 4096 x
    // 8192 140 and 131, 231 and 176.  (Of one piece, 65536 x 512: 122 us so;
    // with biases 131 either way.)
    constexpr bool AHEAD = TPR <= CU_THREADS && !(MANY && V * P == 16);
    uint4 dyn[P], dhn[P], yyn[P], oon[P];
    float stn[4];
    if constexpr (AHEAD) request(it + 1 < turns ? row_of(it + 1) : N, dyn, dhn, yyn, oon, stn);
    const float ry = st[0], my = st[1], ro = st[2], mo = st[3];
    float v[SUMS_ROW];
#pragma unroll
    for (int k = 0; k < SUMS_ROW; ++k) v[k] = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float g[V], x[V], y[V], o[V], c[V], t[V];
      unpack<T>(dh[p], g);
      unpack<T>(w_pre[p], t);
      unpack<T>(yy[p], y);
      unpack<T>(oo[p], o);
      unpack<T>(dy[p], x);
      if constexpr (MANY) {
        float q[V];
        unpack<T>(w_post[p], c);
        unpack<T>(gate[p], q);
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] *= q[i];
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = kw[p][i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // outside the row the weights are zeros: no term counts
        const float yh = (y[i] - my) * ry, oh = (o[i] - mo) * ro, pw = g[i] * t[i];
        const float k = MANY ? A.b * c[i] : c[i], f = x[i] + ry * pw;
        if constexpr (KEPT) kept[(p * V + i) * THREADS + tr] += g[i] * yh;
        else a_wpre[p][i] += g[i] * yh;
        if constexpr (BIAS) a_bpre[p][i] += g[i];
        v[0] += pw * yh;
        v[1] += k * oh * f;
        v[2] += k * oh * yh;
        if constexpr (LAYER) {
          v[3] += pw;
          v[4] += k * oh;
          v[5] += k * f;
          v[6] += k * yh;
          v[7] += k;
        }
      }
    }
    row_sums<TPR, SUMS_ROW, THREADS>(v, lds, half);
    const float m1 = v[0] * inv_h;
    float m2 = 0.f, t1 = 0.f, t2 = 0.f;
    if constexpr (LAYER) m2 = v[3] * inv_h;
    if (A.w_post) {
      t1 = (v[1] - ry * m1 * v[2]) * inv_h;
      if constexpr (LAYER) {
        t1 -= ry * m2 * v[4] * inv_h;
        t2 = (v[5] - ry * (m2 * v[7] + m1 * v[6])) * inv_h;
      }
    }
    if constexpr (AGAIN) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        hold(dy[p]);
        hold(dh[p]);
        hold(yy[p]);
        hold(oo[p]);
        hold(w_post[p]);
        hold(w_pre[p]);
        hold(gate[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float g[V], y[V], o[V], D[V], t[V];
      unpack<T>(dh[p], g);
      unpack<T>(w_pre[p], t);
      unpack<T>(yy[p], y);
      unpack<T>(dy[p], D);
      unpack<T>(oo[p], o);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float yh = (y[i] - my) * ry;
        D[i] += ry * (g[i] * t[i] - m2 - yh * m1);
        o[i] = (o[i] - mo) * ro;
        if (live) {
          if constexpr (KEPT) kept[((P + p) * V + i) * THREADS + tr] += D[i] * o[i];
          else a_1[p][i] += D[i] * o[i];
          if constexpr (BIAS) a_0[p][i] += D[i];
        }
      }
      const int64_t at = (int64_t)n * pieces + tr + p * TPR;
      if (A.O) {
        float q[V];
        if constexpr (MANY) {
          unpack<T>(gate[p], q);
          if (A.w_post) {
            unpack<T>(w_post[p], t);
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = ro * (A.b * q[i] * t[i] * D[i] - t2 - o[i] * t1);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = A.b * q[i] * D[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            q[i] = A.w_post ? ro * (kw[p][i] * D[i] - t2 - o[i] * t1) : kw[p][i] * D[i];
        }
        if (in[p] && live) store_piece<T>(A.dO, at, q);
#pragma unroll
        for (int i = 0; i < V; ++i) D[i] *= A.a;
      }
      if (in[p] && live) store_piece<T>(A.dX, at, D);
    }
    if constexpr (MANY) {
      if (it % per_gate == per_gate - 1) {  // this gate row is done
        const uint32_t g = gate_of(it);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          float q[V], t[V], d[V];
          unpack<T>(gate[p], q);
          unpack<T>(w_post[p], t);
          if (!A.w_post)
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = 1.f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            d[i] = t[i] * a_1[p][i];
            s_1[p][i] += A.b * q[i] * a_1[p][i];
            a_1[p][i] = 0.f;
          }
          if constexpr (BIAS) {
            unpack<T>(A.b_post && in[p] ? load_raw(A.b_post, tr + p * TPR) : zero, t);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              d[i] += t[i] * a_0[p][i];
              s_0[p][i] += A.b * q[i] * a_0[p][i];
              a_0[p][i] = 0.f;
            }
          }
          if (!(in[p] && g < G)) continue;
          const int64_t out = (int64_t)g * A.H + (tr + p * TPR) * V;
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            if (A.accumulate) Store4<float>::load(A.dgate, out + i, o);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += A.b * d[i + j];
            Store4<float>::store(A.dgate, out + i, o);
          }
        }
      }
    }
    if constexpr (AHEAD) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        dy[p] = dyn[p];
        dh[p] = dhn[p];
        yy[p] = yyn[p];
        oo[p] = oon[p];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) st[k] = stn[k];
    } else {
      request(it + 1 < turns ? row_of(it + 1) : N, dy, dh, yy, oo, st);
    }
  }
  // The row groups' sums meet in shared memory, two arrays at a time (64 KiB
  // at most); each group then adds up its share of the columns, in order.
  constexpr int PV = P * V, EACH = THREADS * PV;
  constexpr int SHARE = PV >= R ? PV / R : 1;
  auto out_of = [&](int k) { return A.ws + ((int64_t)k * W + w) * A.H; };
  auto put = [&](int k, int at, float (&acc)[P][V]) {
    if constexpr (R == 1) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (in[p])
#pragma unroll
          for (int i = 0; i < V; i += 4)
            Store4<float>::store(out_of(k), (tr + p * TPR) * V + i, acc[p] + i);
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) lds[at * EACH + (rg * PV + p * V + i) * TPR + tr] = acc[p][i];
    }
  };
  auto add = [&](int k, int at) {
    const int j0 = rg * SHARE, c = tr + j0 / V * TPR;
    if (j0 >= PV || c >= pieces) return;
    float t[SHARE];
#pragma unroll
    for (int j = 0; j < SHARE; ++j) {
      t[j] = lds[at * EACH + (j0 + j) * TPR + tr];
#pragma unroll
      for (int r = 1; r < R; ++r) t[j] += lds[at * EACH + (r * PV + j0 + j) * TPR + tr];
    }
    float* out = out_of(k) + c * V + j0 % V;
    if constexpr (SHARE % 4 == 0) {
#pragma unroll
      for (int j = 0; j < SHARE; j += 4) Store4<float>::store(out, j, t + j);
    } else {
#pragma unroll
      for (int j = 0; j < SHARE; ++j) out[j] = t[j];
    }
  };
  auto finish = [&](bool one, int k1, float (&a1)[P][V], bool two, int k2, float (&a2)[P][V]) {
    if constexpr (R > 1) __syncthreads();
    if (one) put(k1, 0, a1);
    if (two) put(k2, 1, a2);
    if constexpr (R > 1) {
      __syncthreads();
      if (one) add(k1, 0);
      if (two) add(k2, 1);
    }
  };
  const bool pre = A.w_pre != nullptr, block = A.O != nullptr;
  if constexpr (KEPT) {
    float t[P][V];
    for (int k = 0; k < 2; ++k) {
      if (!(k ? block : pre)) continue;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) t[p][i] = kept[((k * P + p) * V + i) * THREADS + tr];
      put(k ? SUM_1 : SUM_W_PRE, 0, t);
    }
  } else if constexpr (MANY) {
    finish(pre, SUM_W_PRE, a_wpre, block, SUM_1, s_1);
    if constexpr (BIAS) finish(pre, SUM_B_PRE, a_bpre, block, SUM_0, s_0);
  } else {
    finish(pre, SUM_W_PRE, a_wpre, block, SUM_1, a_1);
    if constexpr (BIAS) finish(pre, SUM_B_PRE, a_bpre, block, SUM_0, a_0);
  }
}

// The gradients of the weights from the partial sums: 64 columns and 64
// shares of the workers for each workgroup, so that a thread has four loads
// at most, all on their way at once; blockIdx.y is dw_pre, db_pre, dw_post,
// db_post, then (G <= W) the gate's rows g with the workers w = g, g + G, ...
__device__ __forceinline__ void add4(float4& s, const float4& v) {
  s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
}
__device__ __forceinline__ float4 add_lanes(float4 s) {  // over the lanes 16 and 32 apart
  add4(s, make_float4(__shfl_xor(s.x, 16, 64), __shfl_xor(s.y, 16, 64), __shfl_xor(s.z, 16, 64),
                      __shfl_xor(s.w, 16, 64)));
  add4(s, make_float4(__shfl_xor(s.x, 32, 64), __shfl_xor(s.y, 32, 64), __shfl_xor(s.z, 32, 64),
                      __shfl_xor(s.w, 32, 64)));
  return s;
}
constexpr int SHARES = 64;
template <typename T>
__global__ __launch_bounds__(1024) void reduce_kernel(NormBwdArgs A) {
  __shared__ float4 part[2][16][16];
  const int k = blockIdx.y;
  float* out = k == 0 ? A.dw_pre : k == 1 ? A.db_pre : k == 2 ? A.dw_post : k == 3 ? A.db_post
                                                             : A.dgate + (int64_t)(k - 4) * A.H;
  if (!out) return;
  const int lane = threadIdx.x & 15, share = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane * 4;
  const int W = A.workers;
  const bool is_gate = k >= 4;
  // dw_post, db_post: the workers' gate rows are still to be applied
  const bool weigh = (k == 2 || k == 3) && (A.G == 0 || A.G <= W);
  const int first = is_gate ? k - 4 : 0, step = is_gate ? (int)A.G : 1;
  const int slot = k == 0 ? SUM_W_PRE : k == 1 ? SUM_B_PRE : k == 3 ? SUM_0 : SUM_1;
  const bool second = is_gate && A.b_post;  // the gate's other sum
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f), s0 = s;
  if (c < A.H && A.N > 0) {
    const float* in = A.ws + (int64_t)slot * W * A.H + c;
    const float* in0 = A.ws + (int64_t)SUM_0 * W * A.H + c;
    float4 g = make_float4(A.b, A.b, A.b, A.b);
    if (weigh && A.G == 1) {
      float q[4];
      Store4<T>::load(A.gate, c, q);
      g = make_float4(A.b * q[0], A.b * q[1], A.b * q[2], A.b * q[3]);
    }
#pragma unroll 4
    for (int w = first + share * step; w < W; w += SHARES * step) {
      float4 v = *reinterpret_cast<const float4*>(in + (int64_t)w * A.H);
      if (weigh) {
        if (A.G > 1) {
          float q[4];
          Store4<T>::load(A.gate, (int64_t)(w % (int)A.G) * A.H + c, q);
          g = make_float4(A.b * q[0], A.b * q[1], A.b * q[2], A.b * q[3]);
        }
        v.x *= g.x; v.y *= g.y; v.z *= g.z; v.w *= g.w;
      }
      add4(s, v);
      if (second) add4(s0, *reinterpret_cast<const float4*>(in0 + (int64_t)w * A.H));
    }
  }
  s = add_lanes(s);
  if (second) s0 = add_lanes(s0);
  if ((threadIdx.x & 63) < 16) {
    part[0][wave][lane] = s;
    if (second) part[1][wave][lane] = s0;
  }
  __syncthreads();
  if (share != 0 || c >= A.H) return;
  float p[4] = {1.f, 1.f, 1.f, 1.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
  if (is_gate && A.w_post) Store4<T>::load(A.w_post, c, p);
  if (second) Store4<T>::load(A.b_post, c, b);
#pragma unroll
  for (int j = 1; j < 16; ++j) {
    add4(s, part[0][j][lane]);
    if (second) add4(s0, part[1][j][lane]);
  }
  if (is_gate) {
    s.x = A.b * (p[0] * s.x + b[0] * s0.x);
    s.y = A.b * (p[1] * s.y + b[1] * s0.y);
    s.z = A.b * (p[2] * s.z + b[2] * s0.z);
    s.w = A.b * (p[3] * s.w + b[3] * s0.w);
  }
  float4* o = reinterpret_cast<float4*>(out + c);
  if (A.accumulate) add4(s, *o);
  *o = s;
}

__global__ __launch_bounds__(NT) void zero_kernel(float4* p, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)NT + threadIdx.x; i < n; i += gridDim.x * (int64_t)NT)
    p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// workers of one call, with `at_once` rows to a worker's turn: as many as
// there are compute units where each then has a turn and two rows or more
// (bwd and reduction, 200 x 8192 bf16: 16.5 us so, 19.1 with one row or more,
// 18.2 with four; 999 x 1004 fp32 14.0, 15.5 with two turns)
static int workers_for(int64_t N, int64_t G, int at_once) {
  const int64_t least = at_once > 2 ? at_once : 2;
  int64_t w = (N + least - 1) / least;
  if (w > CUS) w = CUS;
  if (w < 1) w = 1;
  if (G > 0 && G <= w) w = w / G * G;
  return (int)w;
}

static unsigned grid_rows(int64_t n) { return (unsigned)(n < 1 ? 1 : (n > 65535 ? 65535 : n)); }

// f(T{}, bool_constant<LAYER>{}) of the descriptor's type and kind
template <typename F>
static hipError_t pick(int kind, int dtype, F&& f) {
  if (dtype == TP_BF16)
    return kind == TP_NORM_LAYER ? f(bf16_t{}, std::true_type{}) : f(bf16_t{}, std::false_type{});
  return kind == TP_NORM_LAYER ? f(0.f, std::true_type{}) : f(0.f, std::false_type{});
}

}  // namespace norm

// f(TPR, P) of the threads a row and pieces a thread that hold `pieces`
// pieces in registers; false: too wide for any.  Narrow rows (a norm of each
// head's channels) share a wavefront: 262144 x 64 bf16 24 us so, 114 with a
// wavefront each, backward 39 and 148; 281330 x 96 42 and 129, 77 and 164.
// WIDEST: threads of the widest rows.  Forward, 2048 x 16384 bf16: 46 us with
// 512 threads, 82 with 1024 (barriers of 16 wavefronts); backward, whose 512
// threads would spill, 393 and 123 us.
template <int WIDEST, typename F>
static bool pick_width(int64_t pieces, F&& f) {
  using std::integral_constant;
  if (pieces <= 8) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (pieces <= 16) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (pieces <= 32) f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (pieces <= 64) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (pieces <= 128) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (pieces <= 256) f(integral_constant<int, 128>{}, integral_constant<int, 2>{});
  else if (pieces <= 512) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (pieces <= 1024) f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  else if (pieces <= 2048) f(integral_constant<int, WIDEST>{}, integral_constant<int, 2048 / WIDEST>{});
  else return false;
  return true;
}

hipError_t norm_fwd_launch(int kind, int dtype, const NormFwdArgs& a, hipStream_t st) {
  using namespace norm;
  if (a.N == 0) return hipSuccess;
  return pick(kind, dtype, [&](auto t, auto layer) {
    using T = decltype(t);
    constexpr bool L = decltype(layer)::value;
    const bool fits = pick_width<512>(a.H / Piece<T>::V, [&](auto tpr, auto p) {
      constexpr int TPR = decltype(tpr)::value, P = decltype(p)::value;
      const int64_t groups = (a.N + Rows<TPR>::AT_ONCE - 1) / Rows<TPR>::AT_ONCE;
      const int64_t most = (int64_t)CUS * CU_THREADS / Rows<TPR>::THREADS;
      hipLaunchKernelGGL((fwd_kernel<T, L, TPR, P>), dim3((unsigned)(groups < most ? groups : most)),
                         dim3(Rows<TPR>::THREADS), 0, st, a);
    });
    if (!fits)
      hipLaunchKernelGGL((fwd_wide_kernel<T, L>), dim3(grid_rows(a.N)), dim3(NT), 0, st, a);
    return hipGetLastError();
  });
}

// 16 wavefronts a workgroup leave too few registers for bf16 rows with more
// sums than two: those take the wide kernels (2048 x 16384: with biases 221 us
// so, 502 with registers spilled; with a gate a token 321, 342; with both 316,
// 762).  fp32 rows hold half the values; with biases or many gate rows they
// spill 11 to 66 registers and are faster all the same (2048 x 8192 with both
// 215 us, 269 in the wide kernels).
static bool two_sums_only(int dtype, int64_t H) {
  return dtype == TP_BF16 && H > norm::CU_THREADS * 2 * norm::Piece<bf16_t>::V;
}

// Whether the backward unpacks the values of bf16 rows again after the row
// sums.  The widest rows: 2048 x 16384 124 us so, 160 without.  Eight sums of
// two pieces a thread (biases, many gate rows): they leave too few registers
// where a gate row is finished, which costs where its tokens are few.  8192 x
// 4096, RMS: 168 us so and 233 without at a gate a token, 147 and 163 at two
// tokens a gate row, 138 and 128 at four, 130 and 111 at eight, 182 and 132 at
// 27.  Elsewhere it costs (65536 x 512 with biases and a gate a token, one
// piece a thread, 157 us so, 132 without; 381 x 6152 with biases 29.6 and 26.6).
constexpr int64_t AGAIN_BELOW = 4;  // tokens of a gate row
template <typename T, int TPR, int P, bool BIAS, bool MANY>
constexpr bool again_pays() {
  return sizeof(T) == 2 && (TPR > norm::CU_THREADS || (BIAS && MANY && P == 2));
}

// workers of a call, and whether its rows fit the registers
static int bwd_workers(int64_t N, int64_t G, int64_t pieces, bool* fits) {
  using namespace norm;
  int w = 0;
  *fits = pick_width<1024>(pieces, [&](auto tpr, auto) {
    w = workers_for(N, G, BwdRows<decltype(tpr)::value>::AT_ONCE);
  });
  return *fits ? w : workers_for(N, G, 1);
}

size_t norm_bwd_workspace(const tp_norm_desc& d) {
  bool fits;
  const size_t w = (size_t)bwd_workers(d.N, d.gate_rows, d.H / (d.dtype == TP_BF16 ? 8 : 4), &fits);
  // (the descriptor does not say whether there are biases: as for wide rows)
  const bool wide = !fits || two_sums_only(d.dtype, d.H);
  return (w * norm::SUMS * (size_t)d.H + (wide ? 2 * (size_t)d.N : 0)) * sizeof(float);
}

hipError_t norm_bwd_launch(int kind, int dtype, NormBwdArgs& a, hipStream_t st) {
  using namespace norm;
  bool fits;
  a.workers = bwd_workers(a.N, a.G, a.H / (dtype == TP_BF16 ? 8 : 4), &fits);
  const bool many = a.G > a.workers;
  // sums without a factor besides them: the biases' gradients, and the
  // gate's where a bias is in its factor
  const bool bias = a.db_pre || a.db_post || (a.b_post && a.dgate);
  if ((bias || many) && two_sums_only(dtype, a.H)) fits = false;
  return pick(kind, dtype, [&](auto t, auto layer) {
    using T = decltype(t);
    constexpr bool L = decltype(layer)::value;
    hipError_t he = hipSuccess;
    const unsigned W = (unsigned)a.workers;
    if (a.N > 0 && fits) {
      pick_width<1024>(a.H / Piece<T>::V, [&](auto tpr, auto p) {
        constexpr int TPR = decltype(tpr)::value, P = decltype(p)::value;
        constexpr int THREADS = BwdRows<TPR>::THREADS, R = BwdRows<TPR>::AT_ONCE;
        const size_t sums = 2 * (THREADS / 64) * (L ? 8 : 3) * sizeof(float);
        const size_t meet = R == 1 ? 0 : 2 * sizeof(float) * THREADS * P * Piece<T>::V;
        const size_t lds = sums > meet ? sums : meet;
        auto launch = [&](auto b, auto m, auto again) {
          hipLaunchKernelGGL((bwd_kernel<T, L, decltype(b)::value, decltype(m)::value, decltype(again)::value, TPR, P>),
                             dim3(W), dim3(THREADS), lds, st, a);
        };
        constexpr std::true_type YES{};
        constexpr std::false_type NO{};
        if constexpr (sizeof(T) == 4 || TPR <= CU_THREADS) {  // see two_sums_only
          constexpr std::bool_constant<again_pays<T, TPR, P, true, true>()> again{};
          if (many && !bias) launch(NO, YES, NO);
          else if (many && a.N < AGAIN_BELOW * a.G) launch(YES, YES, again);
          else if (many) launch(YES, YES, NO);
          else if (bias) launch(YES, NO, NO);
        }
        if (!many && !bias) launch(NO, NO, std::bool_constant<again_pays<T, TPR, P, false, false>()>{});
      });
      he = hipGetLastError();
    } else if (a.N > 0) {
      float* means = a.ws + (size_t)a.workers * SUMS * a.H;
      hipLaunchKernelGGL((bwd_wide_rows_kernel<T, L>), dim3(grid_rows(a.N)), dim3(NT), 0, st, a,
                         means);
      if ((he = hipGetLastError()) != hipSuccess) return he;
      const unsigned cols = (unsigned)((a.H + NT * Piece<T>::V - 1) / (NT * Piece<T>::V));
      hipLaunchKernelGGL((bwd_wide_columns_kernel<T, L>), dim3(cols, W), dim3(NT), 0, st, a, means);
      he = hipGetLastError();
    } else if (many && !a.accumulate) {
      hipLaunchKernelGGL(zero_kernel, dim3(1024), dim3(NT), 0, st,
                         reinterpret_cast<float4*>(a.dgate), a.G * a.H / 4);
      he = hipGetLastError();
    }
    if (he != hipSuccess) return he;
    const unsigned gates = a.dgate && !many ? (unsigned)a.G : 0u;
    hipLaunchKernelGGL((reduce_kernel<T>), dim3((unsigned)((a.H + 63) / 64), 4 + gates), dim3(1024), 0,
                       st, a);
    return hipGetLastError();
  });
}

}  // namespace tpmlp
