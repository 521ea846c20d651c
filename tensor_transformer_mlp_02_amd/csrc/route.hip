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

// One wavefront a token.  Lane i holds the experts i V .. i V + V - 1, so
// that a lane's logits are one load and the lower expert is in the lower
// lane.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool live, float l[V]) {
  const int e0 = lane * V;
  if (V > 1 && E % V == 0) {
    constexpr int BYTES = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;
    constexpr int PER = BYTES / (int)sizeof(T);  // logits of a load
    struct alignas(BYTES) Part { T x[PER]; };
#pragma unroll
    for (int i = 0; i < V; i += PER) {
      Part q;
      const bool there = live && e0 < E;
      if (there) q = *reinterpret_cast<const Part*>(row + e0 + i);
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        float x = -__builtin_huge_valf();
        if (there) {
          if constexpr (sizeof(T) == 2) x = bf16_to_f32(q.x[j]); else x = q.x[j];
        }
        l[i + j] = x;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float x = -__builtin_huge_valf();
      if (live && e0 + i < E) {
        if constexpr (sizeof(T) == 2) x = bf16_to_f32(row[e0 + i]); else x = row[e0 + i];
      }
      l[i] = x;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // NaN compares false
    if (!(l[i] > TP_ROUTE_LOWEST)) l[i] = -__builtin_huge_valf();
    l[i] = fminf(l[i], TP_ROUTE_LARGEST);
  }
}

// Moves within a wavefront that need no shared memory: lane ^ 1, ^ 2, the
// mirror of 8 and of 16 lanes (which bring the other half once the halves
// agree), and lane ^ 16, ^ 32.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int STEP>  // 0..5: over pairs, 4, 8, 16, 32, 64 lanes
__device__ __forceinline__ float other(float x) {
  if constexpr (STEP == 0) return dpp<0xB1>(x);        // quad_perm 1,0,3,2
  else if constexpr (STEP == 1) return dpp<0x4E>(x);   // quad_perm 2,3,0,1
  else if constexpr (STEP == 2) return dpp<0x141>(x);  // row_half_mirror
  else if constexpr (STEP == 3) return dpp<0x140>(x);  // row_mirror
  else if constexpr (STEP == 4) return __shfl_xor(x, 16, 64);
  else return __shfl_xor(x, 32, 64);
}
template <int STEP>
__device__ __forceinline__ double other(double x) {
  const unsigned long long b = __double_as_longlong(x);
  const uint32_t lo = __float_as_uint(other<STEP>(__uint_as_float((uint32_t)b)));
  const uint32_t hi = __float_as_uint(other<STEP>(__uint_as_float((uint32_t)(b >> 32))));
  return __longlong_as_double(((unsigned long long)hi << 32) | lo);
}

// sums and maxima over the wavefront: 16 lanes by moves, then the four rows
// through scalar registers
__device__ __forceinline__ float lane_value(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, other<0>(x));
  x = fmaxf(x, other<1>(x));
  x = fmaxf(x, other<2>(x));
  x = fmaxf(x, other<3>(x));
  return fmaxf(fmaxf(lane_value(x, 0), lane_value(x, 16)),
               fmaxf(lane_value(x, 32), lane_value(x, 48)));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += other<0>(x);
  x += other<1>(x);
  x += other<2>(x);
  x += other<3>(x);
  return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}
__device__ __forceinline__ double wave_sum(double x) {
  x += other<0>(x);
  x += other<1>(x);
  x += other<2>(x);
  x += other<3>(x);
  x += other<4>(x);
  x += other<5>(x);
  return x;
}
__device__ __forceinline__ int wave_sum(int x) {
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

// The largest and second largest of a run of experts, merged over 2^STEPS
// lanes
template <int STEP>
__device__ __forceinline__ void merge_best(double& b1, double& b2) {
  const double o1 = other<STEP>(b1), o2 = other<STEP>(b2);
  b2 = fmax(fmin(b1, o1), fmax(b2, o2));
  b1 = fmax(b1, o1);
}

// Which groups stay, one bit each.  worth: this lane's group's, in lane g.
__device__ __forceinline__ unsigned long long keep_groups(double worth, int groups, int kept,
                                                          int lane) {
  const unsigned long long b = __double_as_longlong(worth);
  int rank = 0;
  for (int g = 0; g < groups; ++g) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, g);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), g);
    const double o = __longlong_as_double(((unsigned long long)hi << 32) | lo);
    rank += o > worth || (o == worth && g < lane);
  }
  return __ballot(lane < groups && rank < kept);
}

// WIDE: scores in 64 bits, where a choice hangs on them (a bias, or groups
// by the sum of two); otherwise the order of the scores is the logits' own.
//
// The k-th choice is a maximum over the wavefront of 32-bit keys: the
// logits, or the choice scores rounded once, which keeps their order but
// for equals.  So k + 1 maxima that all differ settle the choice; where two
// are equal the token is done again on the 64-bit values (tie).
template <typename T, int V, bool SIGMOID, bool WIDE>
__global__ __launch_bounds__(NT) void fwd_kernel(FwdArgs A) {
  extern __shared__ double sh[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* logits = reinterpret_cast<const T*>(A.logits);
  const double NEG = -__builtin_huge_val();
  const float NEGF = -__builtin_huge_valf();
  for (int64_t t = (int64_t)blockIdx.x * WAVES + wave; t < A.N; t += (int64_t)gridDim.x * WAVES) {
    float l[V], s[V], key[V];
    double c[WIDE ? V : 1];
    load_row<T, V>(logits + t * A.E, A.E, lane, true, l);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
    if constexpr (!SIGMOID) top = wave_max(top);
    if constexpr (WIDE) {
      double s64[V], sum = 0.0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (SIGMOID) {
          s64[i] = l[i] > TP_ROUTE_LOWEST ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
        } else {
          s64[i] = l[i] > TP_ROUTE_LOWEST ? exp((double)l[i] - (double)top) : 0.0;
          sum += s64[i];
        }
      }
      if constexpr (!SIGMOID) {
        sum = wave_sum(sum);
        const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) s64[i] *= inv;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        s[i] = (float)s64[i];
        c[i] = s64[i];
        if (A.bias && e < A.E) c[i] += (double)A.bias[e];
        if (!(l[i] > TP_ROUTE_LOWEST)) c[i] = NEG;
        key[i] = A.bias ? (float)c[i] : l[i];
      }
    } else {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (SIGMOID) {
          s[i] = l[i] > TP_ROUTE_LOWEST ? 1.f / (1.f + expf(-l[i])) : 0.f;
        } else {
          s[i] = l[i] > TP_ROUTE_LOWEST ? expf(l[i] - top) : 0.f;
          sum += s[i];
        }
        key[i] = l[i];
      }
      if constexpr (!SIGMOID) {
        sum = wave_sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= inv;
      }
    }
    if (A.groups > 1) {
      const int per = A.E / A.groups;
      double b1 = NEG, b2 = NEG;
      const int lanes = per / V;
      const bool aligned = per % V == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
      if (aligned) {
        // a group is an aligned power of two of whole lanes
#pragma unroll
        for (int i = 0; i < V; ++i) {
          double x;
          if constexpr (WIDE) x = c[i]; else x = (double)key[i];
          b2 = fmax(b2, fmin(b1, x));
          b1 = fmax(b1, x);
        }
        if (lanes > 1) merge_best<0>(b1, b2);
        if (lanes > 2) merge_best<1>(b1, b2);
        if (lanes > 4) merge_best<2>(b1, b2);
        if (lanes > 8) merge_best<3>(b1, b2);
        // lane g takes group g's from the group's first lane
        const double w1 = __shfl(b1, (lane * lanes) & 63, 64), w2 = __shfl(b2, (lane * lanes) & 63, 64);
        b1 = w1;
        b2 = w2;
      } else {
        double* cs = sh + (size_t)wave * A.E;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          double x;
          if constexpr (WIDE) x = c[i]; else x = (double)key[i];
          if (lane * V + i < A.E) cs[lane * V + i] = x;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (lane < A.groups)
          for (int j = 0; j < per; ++j) {
            const double x = cs[lane * per + j];
            b2 = fmax(b2, fmin(b1, x));
            b1 = fmax(b1, x);
          }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      }
      const double worth = A.best == 2 && b2 > NEG ? b1 + b2 : b1;
      const unsigned long long keep = keep_groups(worth, A.groups, A.kept, lane);
      const int mine = aligned ? lane >> (__ffs(lanes) - 1) : 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int g = aligned ? mine : (lane * V + i) / per;
        if (!((keep >> (g & 63)) & 1)) {
          key[i] = NEGF;
          if constexpr (WIDE) c[i] = NEG;
        }
      }
    }
    int my_e = -1;
    float my_s = 0.f;
    // a choice by rounded scores needs one more maximum to show that no two
    // are equal
    const bool check = WIDE && A.bias;
    float k32[V];
#pragma unroll
    for (int i = 0; i < V; ++i) k32[i] = key[i];
    float before = __builtin_huge_valf();
    bool tie = false;
    for (int j = 0; j < A.K + (check ? 1 : 0); ++j) {
      float head = k32[0], hs = s[0];
      int hi = 0;
#pragma unroll
      for (int i = 1; i < V; ++i)
        if (k32[i] > head) {
          head = k32[i];
          hs = s[i];
          hi = i;
        }
      const float m = wave_max(head);
      if (!(m > NEGF)) break;
      if (check && m == before) {
        tie = true;
        break;
      }
      before = m;
      if (j == A.K) break;
      const int win = __ffsll((unsigned long long)__ballot(head == m)) - 1;
      const int e = win * V + __builtin_amdgcn_readlane(hi, win);
      const float sc = lane_value(hs, win);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i == e) k32[i] = NEGF;
      if (lane == j) {
        my_e = e;
        my_s = sc;
      }
    }
    if constexpr (WIDE) {
      if (tie) {
        my_e = -1;
        my_s = 0.f;
        for (int j = 0; j < A.K; ++j) {
          double head = c[0];
          float hs = s[0];
          int hi = 0;
#pragma unroll
          for (int i = 1; i < V; ++i)
            if (c[i] > head) {
              head = c[i];
              hs = s[i];
              hi = i;
            }
          double m = head;
          m = fmax(m, other<0>(m));
          m = fmax(m, other<1>(m));
          m = fmax(m, other<2>(m));
          m = fmax(m, other<3>(m));
          m = fmax(m, other<4>(m));
          m = fmax(m, other<5>(m));
          if (!(m > NEG)) break;
          const int win = __ffsll((unsigned long long)__ballot(head == m)) - 1;
          const int e = win * V + __builtin_amdgcn_readlane(hi, win);
          const float sc = lane_value(hs, win);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (lane * V + i == e) c[i] = NEG;
          if (lane == j) {
            my_e = e;
            my_s = sc;
          }
        }
      }
    }
    if (A.renorm) my_s /= wave_sum(my_s) + 1e-20f;  // lanes past K hold zeros
    if (lane < A.K) {
      A.expert[t * A.K + lane] = my_e;
      A.weight[t * A.K + lane] = my_s * A.scale;
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
// sigmoid: dl = s (1 - s) ds.  One wavefront a token; slot j is lane j's.
template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(NT) void bwd_kernel(BwdArgs A) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t t = (int64_t)blockIdx.x * WAVES + wave; t < A.N; t += (int64_t)gridDim.x * WAVES) {
    const T* row = reinterpret_cast<const T*>(A.logits) + t * A.E;
    int e = -1;
    int64_t r = -1;
    if (lane < A.K) {
      e = A.expert[t * A.K + lane];
      r = A.slot_row ? (int64_t)A.slot_row[t * A.K + lane] : t * A.K + lane;
    }
    float l[V], s[V];
    load_row<T, V>(row, A.E, lane, true, l);
    if (e < 0 || e >= A.E) e = -1;
    float up = 0.f, le = -__builtin_huge_valf();
    if (e >= 0) {
      if (!A.slot_row || (r >= 0 && r < A.R)) up = A.d_weight[r] * A.scale;
      if constexpr (sizeof(T) == 2) le = bf16_to_f32(row[e]); else le = row[e];
    }
    if (!(le > TP_ROUTE_LOWEST)) le = -__builtin_huge_valf();
    le = fminf(le, TP_ROUTE_LARGEST);
    float se;
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = l[i] > TP_ROUTE_LOWEST ? 1.f / (1.f + expf(-l[i])) : 0.f;
      se = le > TP_ROUTE_LOWEST ? 1.f / (1.f + expf(-le)) : 0.f;
    } else {
      float top = l[0], sum = 0.f;
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = wave_max(top);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > TP_ROUTE_LOWEST ? expf(l[i] - top) : 0.f;
        sum += s[i];
      }
      sum = wave_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
      se = le > TP_ROUTE_LOWEST ? expf(le - top) * inv : 0.f;
    }
    float d = up;
    if (A.renorm) {
      const float S = wave_sum(se) + 1e-20f;
      d = (up - wave_sum(up * se / S)) / S;
    }
    if (e < 0) d = 0.f;
    float ds[V];
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] = 0.f;
    // an expert that stands twice counts twice, in slot order
    for (int j = 0; j < A.K; ++j) {
      const int ej = __builtin_amdgcn_readlane(e, j);
      const float dj = lane_value(d, j);
#pragma unroll
      for (int i = 0; i < V; ++i) ds[i] += lane * V + i == ej ? dj : 0.f;
    }
    float dot = 0.f;
    if constexpr (!SIGMOID) dot = wave_sum(d * se);
    T* out = reinterpret_cast<T*>(A.dlogits) + t * A.E;
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] = SIGMOID ? s[i] * (1.f - s[i]) * ds[i] : s[i] * (ds[i] - dot);
    const int e0 = lane * V;
    if (V > 1 && A.E % V == 0) {
      if (e0 < A.E) {
        constexpr int BYTES = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;
        constexpr int PER = BYTES / (int)sizeof(T);
        struct alignas(BYTES) Part { T x[PER]; };
#pragma unroll
        for (int i = 0; i < V; i += PER) {
          Part q;
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            if constexpr (sizeof(T) == 2) q.x[j] = f32_to_bf16(ds[i + j]); else q.x[j] = ds[i + j];
          }
          *reinterpret_cast<Part*>(out + e0 + i) = q;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < A.E) {
          if constexpr (sizeof(T) == 2) out[e0 + i] = f32_to_bf16(ds[i]); else out[e0 + i] = ds[i];
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Dispatch tables: a stable counting sort of the (token, slot) pairs by
// local expert.  A workgroup takes a run of whole tokens, one pair a thread:
// a pair's row is its expert's first row, plus the expert's pairs in earlier
// runs, in earlier wavefronts and in lower lanes.
//   ws: cnt [runs][n_local + 1], pairs of each expert in each run (last: all)
// One run needs no counts of others.  Up to FEW runs, place_kernel adds up
// the earlier runs' counts itself; beyond, scan_kernel turns the counts into
// sums over the earlier runs, and leaves the totals in row `runs`.
// ---------------------------------------------------------------------------
constexpr int RUN = 1024;  // threads of a run
constexpr int FEW = 128;
static int run_tokens(int K) { return RUN / K; }

__device__ __forceinline__ int local_expert(const TablesArgs& A, int64_t f, int64_t f1) {
  if (f >= f1) return -1;
  const int32_t x = A.expert[f];
  return x >= A.first && x - A.first < A.n_local ? x - A.first : -1;
}

__global__ __launch_bounds__(RUN) void count_kernel(TablesArgs A, int pairs) {
  extern __shared__ int hist[];
  const int width = A.n_local + 1;
  for (int e = threadIdx.x; e < width; e += RUN) hist[e] = 0;
  __syncthreads();
  const int64_t f0 = (int64_t)blockIdx.x * pairs, f1 = min(f0 + pairs, A.N * A.K);
  const int e = threadIdx.x < pairs ? local_expert(A, f0 + threadIdx.x, f1) : -1;
  if (e >= 0) atomicAdd(&hist[e], 1);
  const unsigned long long on = __ballot(e >= 0);
  if ((threadIdx.x & 63) == 0) atomicAdd(&hist[A.n_local], (int)__popcll(on));
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += RUN) A.ws[(int64_t)blockIdx.x * width + i] = hist[i];
}

// 64 columns a workgroup, 16 shares of the runs
__global__ __launch_bounds__(RUN) void scan_kernel(TablesArgs A, int runs) {
  __shared__ int part[16][64];
  const int width = A.n_local + 1;
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int each = (runs + 15) / 16, r0 = min(share * each, runs), r1 = min(r0 + each, runs);
  int sum = 0;
  if (e < width)
    for (int r = r0; r < r1; ++r) sum += A.ws[(int64_t)r * width + e];
  part[share][lane] = sum;
  __syncthreads();
  int base = 0;
  for (int i = 0; i < share; ++i) base += part[i][lane];
  if (e >= width) return;
  for (int r = r0; r < r1; ++r) {
    int* p = A.ws + (int64_t)r * width + e;
    const int v = *p;
    *p = base;
    base += v;
  }
  if (share == 15) A.ws[(int64_t)runs * width + e] = base;
}

__global__ __launch_bounds__(RUN) void place_kernel(TablesArgs A, int pairs, int runs) {
  extern __shared__ int lds[];
  const int width = A.n_local + 1;
  int* first = lds;                 // [n_local + 1] first row of each expert in this run
  int* total = first + width;       // [n_local + 1] rows of each expert in all
  int* seen = total + width;        // [RUN] experts of this run's pairs
  int* red = seen + RUN;            // [32]
  uint16_t* waves = reinterpret_cast<uint16_t*>(red + 32);  // [16][n_local] pairs in earlier wavefronts
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int run = blockIdx.x;
  const int64_t f0 = (int64_t)run * pairs, f1 = min(f0 + pairs, A.N * A.K), f = f0 + tid;
  const int e = tid < pairs ? local_expert(A, f, f1) : -1;
  seen[tid] = e;
  for (int i = tid; i < 16 * A.n_local; i += RUN) waves[i] = 0;
  for (int i = tid; i < 2 * width; i += RUN) lds[i] = 0;
  __syncthreads();
  // rank among the lanes with the same expert
  const unsigned long long below = (1ull << lane) - 1;
  const unsigned long long on = __ballot(e >= 0);
  unsigned long long same = on;
  for (int b = 0; (1 << b) < A.n_local; ++b) {
    const unsigned long long bit = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? bit : ~bit;
  }
  const int rank = __popcll(same & below);
  if (e >= 0 && rank == 0) waves[wave * A.n_local + e] = (uint16_t)__popcll(same);
  if (lane == 0) red[wave] = __popcll(on);
  // the other runs
  if (runs > FEW) {
    for (int i = tid; i < width; i += RUN) {
      first[i] = A.ws[(int64_t)run * width + i];
      total[i] = A.ws[(int64_t)runs * width + i];
    }
  } else if (runs > 1) {
    // column by column, the runs dealt to as many threads as there are
    const int shares = max(1, RUN / width);
    for (int i = tid; i < width * shares; i += RUN) {
      const int col = i % width, share = i / width;
      int before = 0, all = 0;
      for (int r = share; r < runs; r += shares) {
        const int v = A.ws[(int64_t)r * width + col];
        all += v;
        before += r < run ? v : 0;
      }
      if (all) atomicAdd(&total[col], all);
      if (before) atomicAdd(&first[col], before);
    }
  }
  __syncthreads();
  // pairs in earlier wavefronts; with one run the sums are the totals
  for (int i = tid; i < A.n_local; i += RUN) {
    int sum = 0;
    for (int w = 0; w < 16; ++w) {
      const int v = waves[w * A.n_local + i];
      waves[w * A.n_local + i] = (uint16_t)sum;
      sum += v;
    }
    if (runs <= 1) total[i] = sum;
  }
  int mine = 0, listed = 0;  // list entries in earlier wavefronts, and of the run
  for (int w = 0; w < 16; ++w) {
    mine += w < wave ? red[w] : 0;
    listed += red[w];
  }
  if (runs <= 1 && tid == 0) total[A.n_local] = listed;
  __syncthreads();
  // first rows: exclusive sums of the totals over the experts (n_local <=
  // RUN: one each)
  {
    const int v = tid < A.n_local ? total[tid] : 0;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(x, d, 64);
      if (lane >= d) x += u;
    }
    if (lane == 63) red[16 + wave] = x;
    __syncthreads();
    int base = x - v;
    for (int w = 0; w < wave; ++w) base += red[16 + w];
    if (tid < A.n_local) {
      first[tid] += base;
      if (run == 0) A.offsets[tid] = base;
    }
  }
  const int rows = total[A.n_local];
  if (run == 0 && tid == 0) {
    A.offsets[A.n_local] = rows;
    A.tok_ptr[A.N] = rows;
  }
  __syncthreads();
  for (int64_t r = rows + (int64_t)run * RUN + tid; r < A.R; r += (int64_t)gridDim.x * RUN) {
    A.row_token[r] = -1;
    A.tok_rows[r] = -1;
    if (A.row_weight) A.row_weight[r] = 0.f;
  }
  if (tid >= pairs || f >= f1) return;
  const int slot = tid % A.K, token0 = tid - slot;
  const int64_t t = (int64_t)run * (pairs / A.K) + tid / A.K;
  // list entries of this token's earlier slots, and of its lower rows
  int earlier = 0, lower = 0;
  for (int i = 0; i < A.K; ++i) {
    const int o = seen[token0 + i];
    if (o < 0) continue;
    earlier += i < slot;
    lower += o < e || (o == e && i < slot);
  }
  const int start = first[A.n_local] + mine + __popcll(on & below) - earlier;
  if (slot == 0) A.tok_ptr[t] = start;
  int row = -1;
  if (e >= 0) {
    row = first[e] + waves[wave * A.n_local + e] + rank;
    A.tok_rows[start + lower] = row;
    A.row_token[row] = (int32_t)t;
    if (A.row_weight) A.row_weight[row] = A.weight[f];
  }
  A.slot_row[f] = row;
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
  const bool wide = bias || (d.groups > 1 && d.group_best == 2);
  return pick(d.dtype, d.E, d.score, [&](auto t, auto v, auto sig) {
    const size_t lds = d.groups > 1 ? (size_t)WAVES * d.E * sizeof(double) : 0;
    const dim3 grid(grid_tokens(d.N));
    if (wide)
      hipLaunchKernelGGL((fwd_kernel<decltype(t), decltype(v)::value, decltype(sig)::value, true>),
                         grid, dim3(NT), lds, st, a);
    else
      hipLaunchKernelGGL((fwd_kernel<decltype(t), decltype(v)::value, decltype(sig)::value, false>),
                         grid, dim3(NT), lds, st, a);
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
                       dim3(grid_tokens(d.N)), dim3(NT), 0, st, a);
    return hipGetLastError();
  });
}

size_t route_tables_workspace(int64_t N, int K, int n_local) {
  const int64_t tokens = route::run_tokens(K);
  const int64_t runs = (N + tokens - 1) / tokens;
  if (runs <= 1) return 16;  // not used; a caller need not tell sizes apart
  return (size_t)(runs + (runs > route::FEW ? 1 : 0)) * ((size_t)n_local + 1) * sizeof(int32_t);
}

hipError_t route_tables_launch(const TablesArgs& a, hipStream_t st) {
  using namespace route;
  const int tokens = run_tokens(a.K), pairs = tokens * a.K;
  const int runs = (int)((a.N + tokens - 1) / tokens);
  const size_t width = (size_t)a.n_local + 1;
  hipError_t he = hipSuccess;
  if (runs > 1) {
    hipLaunchKernelGGL(count_kernel, dim3((unsigned)runs), dim3(RUN), width * sizeof(int), st, a, pairs);
    if ((he = hipGetLastError()) != hipSuccess) return he;
  }
  if (runs > FEW) {
    hipLaunchKernelGGL(scan_kernel, dim3((unsigned)((width + 63) / 64)), dim3(RUN), 0, st, a, runs);
    if ((he = hipGetLastError()) != hipSuccess) return he;
  }
  const size_t lds = (2 * width + RUN + 32) * sizeof(int) + 16 * (size_t)a.n_local * sizeof(uint16_t);
  hipLaunchKernelGGL(place_kernel, dim3((unsigned)(runs > 0 ? runs : 1)), dim3(RUN), lds, st, a,
                     pairs, runs);
  return hipGetLastError();
}

}  // namespace tpmlp
