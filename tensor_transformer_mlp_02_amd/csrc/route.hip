// Routing of tokens to experts (Megatron Core 带读 §09: router -> top-k
// experts -> tokens sent to their experts): scores, the choice of the top k
// within the groups kept, its weights, the logits' gradient, and the
// dispatch tables that the permute / combine kernels and the grouped
// products with device-resident offsets read.
#include "block_launch.h"
#include "common.h"

namespace tpmlp {
namespace route {

constexpr int NT = 256;
constexpr int WAVES = NT / 64;
// a logit at or below the lowest finite bf16 (or NaN) is no choice
#define TP_ROUTE_LOWEST (-3.3895313892515355e38f)
#define TP_ROUTE_LARGEST 3.4028234663852886e38f

template <typename T> __device__ __forceinline__ float load_logit(const T* p, int64_t i);
template <> __device__ __forceinline__ float load_logit<float>(const float* p, int64_t i) {
  return p[i];
}
template <> __device__ __forceinline__ float load_logit<bf16_t>(const bf16_t* p, int64_t i) {
  return bf16_to_f32(p[i]);
}
__device__ __forceinline__ void store_logit(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_logit(bf16_t* p, int64_t i, float v) { p[i] = f32_to_bf16(v); }

template <typename X>
__device__ __forceinline__ X wave_max(X x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const X o = __shfl_xor(x, d, 64);
    x = o > x ? o : x;
  }
  return x;
}
template <typename X>
__device__ __forceinline__ X wave_sum(X x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor(x, d, 64);
  return x;
}

struct FwdArgs {
  const void* logits;
  const float* bias;
  int32_t* expert;
  float* weight;
  int64_t N;
  int E, K, groups, kept, best, renorm;
  float scale;
};

// One wavefront a token, expert e in lane e % 64; choices in 64 bits.
template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(NT) void fwd_kernel(FwdArgs A) {
  extern __shared__ double sh[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double* cs = sh + (size_t)wave * A.E;
  const T* logits = reinterpret_cast<const T*>(A.logits);
  const double NEG = -__builtin_huge_val();
  const int64_t rounds = (A.N + (int64_t)gridDim.x * WAVES - 1) / ((int64_t)gridDim.x * WAVES);
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t t = (it * gridDim.x + blockIdx.x) * WAVES + wave;
    const bool live = t < A.N;
    float l[V];
    double s[V], key[V];
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      float x = live && e < A.E ? load_logit<T>(logits, t * A.E + e) : -__builtin_huge_valf();
      if (!(x > TP_ROUTE_LOWEST)) x = -__builtin_huge_valf();
      l[i] = fminf(x, TP_ROUTE_LARGEST);
      top = fmaxf(top, l[i]);
    }
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        s[i] = l[i] > TP_ROUTE_LOWEST ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
    } else {
      top = wave_max(top);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > TP_ROUTE_LOWEST ? exp((double)l[i] - (double)top) : 0.0;
        sum += s[i];
      }
      sum = wave_sum(sum);
      const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      const bool there = l[i] > TP_ROUTE_LOWEST;
      double c = s[i];
      if (A.bias && e < A.E) c += (double)A.bias[e];
      key[i] = !there ? NEG : A.bias ? c : (double)l[i];
      if (A.groups > 1 && e < A.E) cs[e] = there ? c : NEG;
    }
    if (A.groups > 1) {
      __syncthreads();
      const int per = A.E / A.groups;
      double worth = NEG;
      if (lane < A.groups) {
        double b1 = NEG, b2 = NEG;
        for (int j = 0; j < per; ++j) {
          const double c = cs[lane * per + j];
          if (c > b1) { b2 = b1; b1 = c; } else if (c > b2) { b2 = c; }
        }
        worth = A.best == 2 && b2 > NEG ? b1 + b2 : b1;
      }
      __syncthreads();
      int rank = 0;
      for (int g = 0; g < A.groups; ++g) {
        const double o = __shfl(worth, g, 64);
        rank += o > worth || (o == worth && g < lane);
      }
      const unsigned long long keep = __ballot(lane < A.groups && rank < A.kept);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        if (e < A.E && !((keep >> (e / per)) & 1)) key[i] = NEG;
      }
    }
    // k rounds: the largest key, the lowest expert among equals
    int my_e = -1;
    double my_s = 0.0;
    for (int j = 0; j < A.K; ++j) {
      double m = NEG;
#pragma unroll
      for (int i = 0; i < V; ++i) m = key[i] > m ? key[i] : m;
      m = wave_max(m);
      int at = 0x7fffffff;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (key[i] == m && m > NEG) at = lane + 64 * i;
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) at = min(at, __shfl_xor(at, d, 64));
      const bool none = at == 0x7fffffff;
      double sc = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 64 * i == at) {
          sc = s[i];
          key[i] = NEG;
        }
      sc = __shfl(sc, at & 63, 64);
      if (lane == j) {
        my_e = none ? -1 : at;
        my_s = none ? 0.0 : sc;
      }
    }
    if (A.renorm) my_s /= wave_sum(lane < A.K ? my_s : 0.0) + 1e-20;
    if (live && lane < A.K) {
      A.expert[t * A.K + lane] = my_e;
      A.weight[t * A.K + lane] = (float)(my_s * (double)A.scale);
    }
  }
}

struct BwdArgs {
  const void* logits;
  const int32_t* expert;
  const float* d_weight;
  const int32_t* slot_row;
  void* dlogits;
  int64_t N, R;
  int E, K, renorm;
  float scale;
};

// t_j = scale dw_j; renorm: ds_j = (t_j - sum_i t_i s_i / S) / S with
// S = sum s + 1e-20, else ds_j = t_j; then softmax: dl = s (ds - sum ds s),
// sigmoid: dl = s (1 - s) ds.  One wavefront a token.
template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(NT) void bwd_kernel(BwdArgs A) {
  extern __shared__ float shf[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* ss = shf + (size_t)wave * 2 * A.E;
  float* ds = ss + A.E;
  const T* logits = reinterpret_cast<const T*>(A.logits);
  T* out = reinterpret_cast<T*>(A.dlogits);
  const int64_t rounds = (A.N + (int64_t)gridDim.x * WAVES - 1) / ((int64_t)gridDim.x * WAVES);
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t t = (it * gridDim.x + blockIdx.x) * WAVES + wave;
    const bool live = t < A.N;
    float l[V], s[V];
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      float x = live && e < A.E ? load_logit<T>(logits, t * A.E + e) : -__builtin_huge_valf();
      if (!(x > TP_ROUTE_LOWEST)) x = -__builtin_huge_valf();
      l[i] = fminf(x, TP_ROUTE_LARGEST);
      top = fmaxf(top, l[i]);
    }
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = l[i] > TP_ROUTE_LOWEST ? 1.f / (1.f + expf(-l[i])) : 0.f;
    } else {
      top = wave_max(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > TP_ROUTE_LOWEST ? expf(l[i] - top) : 0.f;
        sum += s[i];
      }
      sum = wave_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      if (e < A.E) {
        ss[e] = s[i];
        ds[e] = 0.f;
      }
    }
    __syncthreads();
    int e = -1;
    float up = 0.f;
    if (live && lane < A.K) {
      e = A.expert[t * A.K + lane];
      if (e < 0 || e >= A.E) e = -1;
      if (A.slot_row) {
        const int32_t r = A.slot_row[t * A.K + lane];
        up = r >= 0 && r < A.R ? A.d_weight[r] : 0.f;
      } else {
        up = A.d_weight[t * A.K + lane];
      }
      up = e < 0 ? 0.f : up * A.scale;
    }
    const float se = e >= 0 ? ss[e] : 0.f;
    float d = up;
    if (A.renorm) {
      const float S = wave_sum(se) + 1e-20f;
      d = (up - wave_sum(up * se / S)) / S;
    }
    if (e < 0) d = 0.f;
    // an expert that stands twice counts twice: each of its slots writes the
    // same sum, taken in slot order
    float all = 0.f;
    for (int j = 0; j < A.K; ++j) {
      const int ej = __shfl(e, j, 64);
      const float dj = __shfl(d, j, 64);
      if (ej == e) all += dj;
    }
    if (e >= 0) ds[e] = all;
    __syncthreads();
    float dot = 0.f;
    if constexpr (!SIGMOID) dot = wave_sum(d * se);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int x = lane + 64 * i;
      if (x < A.E && live) {
        const float g = SIGMOID ? s[i] * (1.f - s[i]) * ds[x] : s[i] * (ds[x] - dot);
        store_logit(out, t * A.E + x, g);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Dispatch tables: a stable counting sort of the (token, slot) pairs by
// local expert.  A wavefront takes a run of whole tokens (`run` pairs): it
// counts its pairs for each expert (count_kernel), scan_kernel turns the
// counts, expert by expert and run by run, into each run's first row of
// each expert, and place_kernel deals the rows out.
//   ws: cnt [n_local][runs], tok [runs]
// ---------------------------------------------------------------------------
constexpr int RUN = 256;  // pairs of a run, at most
static int run_tokens(int K) { return RUN / K; }

__global__ __launch_bounds__(64) void count_kernel(TablesArgs A, int tokens, int runs) {
  extern __shared__ int hist[];
  const int run = blockIdx.x, lane = threadIdx.x;
  for (int e = lane; e < A.n_local; e += 64) hist[e] = 0;
  __syncthreads();
  const int64_t f0 = (int64_t)run * tokens * A.K;
  const int64_t f1 = min(f0 + (int64_t)tokens * A.K, A.N * A.K);
  int mine = 0;
  for (int64_t f = f0 + lane; f < f1; f += 64) {
    const int32_t x = A.expert[f];
    if (x >= A.first && x - A.first < A.n_local) {
      atomicAdd(&hist[x - A.first], 1);
      ++mine;
    }
  }
  __syncthreads();
  for (int e = lane; e < A.n_local; e += 64) A.ws[(int64_t)e * runs + run] = hist[e];
  mine = wave_sum(mine);
  if (lane == 0) A.ws[(int64_t)A.n_local * runs + run] = mine;
}

// exclusive sums of one array of `n` ints in place by one workgroup;
// returns the total
__device__ int block_exclusive(int* a, int64_t n, int* red) {
  int carry = 0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t i0 = 0; i0 < n; i0 += 1024) {
    const int64_t i = i0 + threadIdx.x;
    const int v = i < n ? a[i] : 0;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(x, d, 64);
      if (lane >= d) x += u;
    }
    if (lane == 63) red[wave] = x;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? red[w] : 0;
      all += red[w];
    }
    if (i < n) a[i] = before + x - v;
    carry += all;
    __syncthreads();
  }
  return carry;
}

// workgroup 0: rows (all experts' runs in order) and the offsets;
// workgroup 1: the tokens' lists
__global__ __launch_bounds__(1024) void scan_kernel(TablesArgs A, int runs) {
  __shared__ int red[16];
  if (blockIdx.x == 0) {
    const int total = block_exclusive(A.ws, (int64_t)A.n_local * runs, red);
    __syncthreads();
    for (int e = threadIdx.x; e < A.n_local; e += 1024)
      A.offsets[e] = runs > 0 ? A.ws[(int64_t)e * runs] : 0;
    if (threadIdx.x == 0) A.offsets[A.n_local] = total;
  } else {
    const int total = block_exclusive(A.ws + (int64_t)A.n_local * runs, runs, red);
    if (threadIdx.x == 0) A.tok_ptr[A.N] = total;
  }
}

__global__ __launch_bounds__(64) void place_kernel(TablesArgs A, int tokens, int runs) {
  extern __shared__ int next[];
  const int run = blockIdx.x, lane = threadIdx.x;
  // rows past the last one
  const int64_t total = A.tok_ptr[A.N];
  for (int64_t r = total + (int64_t)run * 64 + lane; r < A.R; r += (int64_t)gridDim.x * 64) {
    A.row_token[r] = -1;
    A.tok_rows[r] = -1;
    if (A.row_weight) A.row_weight[r] = 0.f;
  }
  if (run >= runs) return;
  for (int e = lane; e < A.n_local; e += 64) next[e] = A.ws[(int64_t)e * runs + run];
  __syncthreads();
  int before = A.ws[(int64_t)A.n_local * runs + run];  // list entries of earlier tokens
  const int64_t f0 = (int64_t)run * tokens * A.K;
  const int64_t f1 = min(f0 + (int64_t)tokens * A.K, A.N * A.K);
  const unsigned long long below = (1ull << lane) - 1;
  for (int64_t base = f0; base < f1; base += 64) {
    const int64_t f = base + lane;
    int e = -1;
    if (f < f1) {
      const int32_t x = A.expert[f];
      if (x >= A.first && x - A.first < A.n_local) e = x - A.first;
    }
    // the lanes with the same expert
    const unsigned long long on = __ballot(e >= 0);
    unsigned long long same = on;
    for (int b = 0; (1 << b) < A.n_local; ++b) {
      const unsigned long long bit = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? bit : ~bit;
    }
    int row = -1;
    if (e >= 0) row = next[e] + __popcll(same & below);
    __syncthreads();
    if (e >= 0 && !(same & ~below & ~(1ull << lane))) next[e] = row + 1;
    __syncthreads();
    if (f < f1) {
      const int64_t t = f / A.K;
      const int j = (int)(f - t * A.K);
      A.slot_row[f] = row;
      // list entries of earlier slots of this token, and of lower rows
      int earlier = 0, lower = 0;
      for (int i = 0; i < A.K; ++i) {
        const int32_t x = A.expert[t * A.K + i];
        if (x < A.first || x - A.first >= A.n_local) continue;
        const int o = x - A.first;
        earlier += i < j;
        lower += o < e || (o == e && i < j);
      }
      const int start = before + __popcll(on & below) - earlier;
      if (j == 0) A.tok_ptr[t] = start;
      if (row >= 0) {
        A.tok_rows[start + lower] = row;
        A.row_token[row] = (int32_t)t;
        if (A.row_weight) A.row_weight[row] = A.weight[f];
      }
    }
    before += __popcll(on);
  }
}

template <typename F>
static hipError_t pick(int dtype, int E, int score, F&& f) {
  auto by_score = [&](auto t, auto v) {
    return score == TP_SCORE_SIGMOID ? f(t, v, std::true_type{}) : f(t, v, std::false_type{});
  };
  auto by_size = [&](auto t) {
    if (E <= 64) return by_score(t, std::integral_constant<int, 1>{});
    if (E <= 128) return by_score(t, std::integral_constant<int, 2>{});
    if (E <= 256) return by_score(t, std::integral_constant<int, 4>{});
    if (E <= 512) return by_score(t, std::integral_constant<int, 8>{});
    return by_score(t, std::integral_constant<int, 16>{});
  };
  return dtype == TP_BF16 ? by_size(bf16_t{}) : by_size(0.f);
}

static unsigned grid_tokens(int64_t N) {
  const int64_t b = (N + WAVES - 1) / WAVES;
  return (unsigned)(b > 8192 ? 8192 : b);
}

}  // namespace route

hipError_t route_fwd_launch(const tp_route_desc& d, const void* logits, const float* bias,
                            int32_t* expert, float* weight, hipStream_t st) {
  using namespace route;
  if (d.N == 0) return hipSuccess;
  FwdArgs a{logits, bias, expert, weight, d.N, d.E, d.K, d.groups, d.groups_kept, d.group_best,
            d.renorm, d.scale};
  return pick(d.dtype, d.E, d.score, [&](auto t, auto v, auto sig) {
    const size_t lds = d.groups > 1 ? (size_t)WAVES * d.E * sizeof(double) : 0;
    hipLaunchKernelGGL((fwd_kernel<decltype(t), decltype(v)::value, decltype(sig)::value>),
                       dim3(grid_tokens(d.N)), dim3(NT), lds, st, a);
    return hipGetLastError();
  });
}

hipError_t route_bwd_launch(const tp_route_desc& d, const void* logits, const int32_t* expert,
                            const float* d_weight, const int32_t* slot_row, int64_t R,
                            void* dlogits, hipStream_t st) {
  using namespace route;
  if (d.N == 0) return hipSuccess;
  BwdArgs a{logits, expert, d_weight, slot_row, dlogits, d.N, R, d.E, d.K, d.renorm, d.scale};
  return pick(d.dtype, d.E, d.score, [&](auto t, auto v, auto sig) {
    hipLaunchKernelGGL((bwd_kernel<decltype(t), decltype(v)::value, decltype(sig)::value>),
                       dim3(grid_tokens(d.N)), dim3(NT), (size_t)WAVES * 2 * d.E * sizeof(float),
                       st, a);
    return hipGetLastError();
  });
}

size_t route_tables_workspace(int64_t N, int K, int n_local) {
  const int64_t tokens = route::run_tokens(K);
  const int64_t runs = (N + tokens - 1) / tokens;
  return (size_t)(runs * ((int64_t)n_local + 1)) * sizeof(int32_t);
}

hipError_t route_tables_launch(const TablesArgs& a, hipStream_t st) {
  using namespace route;
  const int tokens = run_tokens(a.K);
  const int runs = (int)((a.N + tokens - 1) / tokens);
  const size_t lds = (size_t)a.n_local * sizeof(int);
  hipError_t he = hipSuccess;
  if (runs > 0) {
    hipLaunchKernelGGL(count_kernel, dim3((unsigned)runs), dim3(64), lds, st, a, tokens, runs);
    if ((he = hipGetLastError()) != hipSuccess) return he;
  }
  hipLaunchKernelGGL(scan_kernel, dim3(2), dim3(1024), 0, st, a, runs);
  if ((he = hipGetLastError()) != hipSuccess) return he;
  if (runs > 0 || a.R > 0) {
    hipLaunchKernelGGL(place_kernel, dim3((unsigned)(runs > 0 ? runs : 64)), dim3(64), lds, st, a,
                       tokens, runs);
    he = hipGetLastError();
  }
  return he;
}

}  // namespace tpmlp
