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
//           starting at w / G; its gate sum is a partial one
//   G > W:  worker w takes the gate rows w, w + W, ... with all their
//           tokens; it finishes each by itself
// (W is rounded down to a multiple of G in the first case.)  The partial
// sums [5][W][H] are added over w, in order, by reduce_kernel.
// ---------------------------------------------------------------------------
enum { SUM_W_PRE = 0, SUM_B_PRE = 1, SUM_W_POST = 2, SUM_B_POST = 3, SUM_GATE = 4, SUMS = 5 };

template <typename Row, typename Flush>
__device__ __forceinline__ void deal_rows(int64_t N, int64_t G, int w, int W, Row&& row,
                                          Flush&& flush) {
  if (G <= W) {
    const int64_t P = W / G;
    for (int64_t n = w % G + (w / G) * G; n < N; n += P * G) row(n);
    flush(-1);
  } else {
    for (int64_t g = w; g < G; g += W) {
      for (int64_t n = g; n < N; n += G) row(n);
      flush(g);
    }
  }
}

template <typename T, bool LAYER>
__global__ __launch_bounds__(NT) void bwd_wide_columns_kernel(NormBwdArgs A, const float* means) {
  constexpr int V = Piece<T>::V;
  const int c = (blockIdx.x * NT + threadIdx.x) * V;
  if (c >= A.H) return;
  const int w = blockIdx.y;
  const int64_t G = A.G > 0 ? A.G : 1;
  float acc[SUMS][V];
#pragma unroll
  for (int k = 0; k < SUMS; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
  float wpost[V], bpost[V];
#pragma unroll
  for (int i = 0; i < V; ++i) { wpost[i] = 1.f; bpost[i] = 0.f; }
  if (A.w_post) Piece<T>::load(A.w_post, c, wpost);
  if (A.b_post) Piece<T>::load(A.b_post, c, bpost);
  deal_rows(
      A.N, G, w, A.workers,
      [&](int64_t n) {
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
        float o[V], g[V];
        Piece<T>::load(A.O, row + c, o);
        if (A.w_post) {
          ro = A.stat_post[n];
          if constexpr (LAYER) mo = A.stat_post[A.N + n];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = 1.f;
        if (A.G > 0) Piece<T>::load(A.gate, (n % A.G) * A.H + c, g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float oh = (o[i] - mo) * ro;
          const float du = A.b * g[i] * D[i];
          acc[SUM_W_POST][i] += du * oh;
          acc[SUM_B_POST][i] += du;
          acc[SUM_GATE][i] += A.b * D[i] * (oh * wpost[i] + bpost[i]);
        }
      },
      [&](int64_t g) {
        if (g < 0 || !A.dgate) return;
        float* out = A.dgate + g * A.H + c;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          out[i] = acc[SUM_GATE][i] + (A.accumulate ? out[i] : 0.f);
          acc[SUM_GATE][i] = 0.f;
        }
      });
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
    if (k == SUM_GATE && (G > A.workers || !A.dgate)) continue;
    float* out = A.ws + ((int64_t)k * A.workers + w) * A.H + c;
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = acc[k][i];
  }
}

// out[c] (+)= sum over the workers, 64 columns and 16 shares of the workers
// for each workgroup; the gate's rows g take the workers w = g, g + G, ...
__global__ __launch_bounds__(NT) void reduce_kernel(NormBwdArgs A, int has_rows) {
  __shared__ float4 part[NT];
  int k = blockIdx.y;
  int first = 0, step = 1;
  float* out;
  if (k < SUM_GATE) {
    out = k == SUM_W_PRE ? A.dw_pre : k == SUM_B_PRE ? A.db_pre : k == SUM_W_POST ? A.dw_post
                                                                               : A.db_post;
  } else {
    first = k - SUM_GATE;
    step = (int)A.G;
    k = SUM_GATE;
    out = A.dgate ? A.dgate + (int64_t)first * A.H : nullptr;
  }
  if (!out) return;
  const int lane = threadIdx.x & 15, share = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + lane * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < A.H && has_rows) {
    const float* in = A.ws + (int64_t)k * A.workers * A.H + c;
    for (int64_t w = first + (int64_t)share * step; w < A.workers; w += 16 * (int64_t)step) {
      const float4 v = *reinterpret_cast<const float4*>(in + w * A.H);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  part[threadIdx.x] = s;
  __syncthreads();
  if (share == 0 && c < A.H) {
#pragma unroll
    for (int j = 1; j < 16; ++j) {
      const float4 v = part[j * 16 + lane];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    float4* o = reinterpret_cast<float4*>(out + c);
    if (A.accumulate) {
      const float4 v = *o;
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    *o = s;
  }
}

__global__ __launch_bounds__(NT) void zero_kernel(float4* p, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)NT + threadIdx.x; i < n; i += gridDim.x * (int64_t)NT)
    p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// workers of one call: enough to fill the chip, at least 4 rows each
static int workers_for(int64_t N, int64_t G) {
  int64_t w = N / 4;
  if (w > 256) w = 256;
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

hipError_t norm_fwd_launch(int kind, int dtype, const NormFwdArgs& a, hipStream_t st) {
  using namespace norm;
  if (a.N == 0) return hipSuccess;
  return pick(kind, dtype, [&](auto t, auto layer) {
    using T = decltype(t);
    hipLaunchKernelGGL((fwd_wide_kernel<T, decltype(layer)::value>), dim3(grid_rows(a.N)),
                       dim3(NT), 0, st, a);
    return hipGetLastError();
  });
}

size_t norm_bwd_workspace(const tp_norm_desc& d) {
  const size_t w = (size_t)norm::workers_for(d.N, d.gate_rows);
  return (w * norm::SUMS * (size_t)d.H + 2 * (size_t)d.N) * sizeof(float);
}

hipError_t norm_bwd_launch(int kind, int dtype, NormBwdArgs& a, hipStream_t st) {
  using namespace norm;
  a.workers = workers_for(a.N, a.G);
  if (a.N > 0) {
    hipError_t he = pick(kind, dtype, [&](auto t, auto layer) {
      using T = decltype(t);
      constexpr bool L = decltype(layer)::value;
      float* means = a.ws + (size_t)a.workers * SUMS * a.H;
      hipLaunchKernelGGL((bwd_wide_rows_kernel<T, L>), dim3(grid_rows(a.N)), dim3(NT), 0, st, a,
                         means);
      hipError_t he = hipGetLastError();
      if (he != hipSuccess) return he;
      const unsigned cols = (unsigned)((a.H + NT * Piece<T>::V - 1) / (NT * Piece<T>::V));
      hipLaunchKernelGGL((bwd_wide_columns_kernel<T, L>), dim3(cols, (unsigned)a.workers),
                         dim3(NT), 0, st, a, means);
      return hipGetLastError();
    });
    if (he != hipSuccess) return he;
  }
  const bool gate_partial = a.dgate && a.G <= a.workers;
  if (a.N == 0 && a.dgate && !gate_partial && !a.accumulate) {
    hipLaunchKernelGGL(zero_kernel, dim3(1024), dim3(NT), 0, st,
                       reinterpret_cast<float4*>(a.dgate), a.G * a.H / 4);
    hipError_t he = hipGetLastError();
    if (he != hipSuccess) return he;
  }
  hipLaunchKernelGGL(reduce_kernel,
                     dim3((unsigned)((a.H + 63) / 64), SUM_GATE + (gate_partial ? (unsigned)a.G : 0u)),
                     dim3(NT), 0, st, a, a.N > 0 ? 1 : 0);
  return hipGetLastError();
}

}  // namespace tpmlp
