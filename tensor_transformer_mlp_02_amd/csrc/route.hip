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
constexpr float LOWEST = -3.3895313892515355e38f;
constexpr float LARGEST = 3.4028234663852886e38f;

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
    if (!(l[i] > LOWEST)) l[i] = -__builtin_huge_valf();
    l[i] = fminf(l[i], LARGEST);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* row, int E, int lane, const float (&g)[V]) {
  const int e0 = lane * V;
  if (V > 1 && E % V == 0) {
    if (e0 >= E) return;
    constexpr int BYTES = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;
    constexpr int PER = BYTES / (int)sizeof(T);
    struct alignas(BYTES) Part { T x[PER]; };
#pragma unroll
    for (int i = 0; i < V; i += PER) {
      Part q;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if constexpr (sizeof(T) == 2) q.x[j] = f32_to_bf16(g[i + j]); else q.x[j] = g[i + j];
      }
      *reinterpret_cast<Part*>(row + e0 + i) = q;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) {
        if constexpr (sizeof(T) == 2) row[e0 + i] = f32_to_bf16(g[i]); else row[e0 + i] = g[i];
      }
  }
}

// Shared memory that one wavefront writes and reads by itself: its accesses
// are in order, the compiler has to keep them so.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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

struct FwdArgs {
  const void* logits;
  const float* bias;
  int32_t* expert;
  float* weight;
  int64_t N;
  int E, K, groups, kept, best, renorm;
  float scale;
  // groups: experts of one; whole lanes of one as a power of two (-1: it is
  // none); x / per = x magic >> 20 for x < 1024
  int per, lanes_log2;
  uint32_t magic;
  int wide_log2;  // lanes_log2 of the 64-bit choice
};

// Keys in unsigned integers that order like the floats, 0 for an expert that
// is not there: maxima need no canonical NaNs, and equal bits are equal keys.
__device__ __forceinline__ uint32_t to_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 is 0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t key_of_lane(uint32_t x, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max_with<0xB1>(x);
  x = max_with<0x4E>(x);
  x = max_with<0x141>(x);
  x = max_with<0x140>(x);
  return max(max(key_of_lane(x, 0), key_of_lane(x, 16)), max(key_of_lane(x, 32), key_of_lane(x, 48)));
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const unsigned long long b = __double_as_longlong(x);
  return __longlong_as_double(((unsigned long long)key_of_lane((uint32_t)(b >> 32), lane) << 32) |
                              key_of_lane((uint32_t)b, lane));
}
__device__ __forceinline__ double wave_max(double x) {
  x = fmax(x, other<0>(x));
  x = fmax(x, other<1>(x));
  x = fmax(x, other<2>(x));
  x = fmax(x, other<3>(x));
  return fmax(fmax(lane_value(x, 0), lane_value(x, 16)), fmax(lane_value(x, 32), lane_value(x, 48)));
}

// The largest and second largest of a run of experts, merged over lanes
template <int STEP, typename X>
__device__ __forceinline__ void merge_best(X& b1, X& b2) {
  const X o1 = other<STEP>(b1), o2 = other<STEP>(b2);
  b2 = fmax(fmin(b1, o1), fmax(b2, o2));
  b1 = fmax(b1, o1);
}

// What a group of experts is worth by its two largest choice scores (-inf: not
// there): the larger one, or half the sum of both (a sum of two finite scores
// may not be finite, and halving rounds nothing that counts).
template <typename X>
__device__ __forceinline__ X worth_of(X b1, X b2, int best) {
  if (best == 1) return b1;
  return (X)0.5 * b1 + (b2 > (X)-__builtin_huge_val() ? (X)0.5 * b2 : (X)0);
}
// The magnitude of its terms, which the worth's rounding goes by: scores of
// opposite signs cancel in the sum, not in its error.
__device__ __forceinline__ float terms_of(float b1, float b2, int best) {
  if (!(b1 > -__builtin_huge_valf())) return 0.f;
  return best == 1 ? fabsf(b1) : worth_of(fabsf(b1), b2 > -__builtin_huge_valf() ? fabsf(b2) : b2, best);
}

// What lane g's group of experts is worth (-inf: none there), and where
// `terms` is given their magnitude.  `cs`: E values of shared memory.
template <typename X, int V>
__device__ __forceinline__ X group_worth(const X (&c)[V], const FwdArgs& A, int lane, X* cs,
                                         float* terms = nullptr) {
  const X NEG = (X)-__builtin_huge_val();
  X b1 = NEG, b2 = NEG;
  if (A.lanes_log2 >= 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b2 = fmax(b2, fmin(b1, c[i]));
      b1 = fmax(b1, c[i]);
    }
    if (A.lanes_log2 > 0) merge_best<0>(b1, b2);
    if (A.lanes_log2 > 1) merge_best<1>(b1, b2);
    if (A.lanes_log2 > 2) merge_best<2>(b1, b2);
    if (A.lanes_log2 > 3) merge_best<3>(b1, b2);
    const int from = (lane << A.lanes_log2) & 63;
    if (terms) *terms = __shfl(terms_of((float)b1, (float)b2, A.best), from, 64);
    return __shfl(worth_of(b1, b2, A.best), from, 64);
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (lane * V + i < A.E) cs[lane * V + i] = c[i];
  wave_lds_sync();
  if (lane < A.groups)
    for (int j = 0; j < A.per; ++j) {
      const X x = cs[lane * A.per + j];
      b2 = fmax(b2, fmin(b1, x));
      b1 = fmax(b1, x);
    }
  wave_lds_sync();
  if (terms) *terms = terms_of((float)b1, (float)b2, A.best);
  return worth_of(b1, b2, A.best);
}

// Which groups stay, one bit each: the `kept` worth most, the lower of equals
template <typename X>
__device__ __forceinline__ unsigned long long keep_groups(X worth, const FwdArgs& A, int lane) {
  int rank = 0;
  for (int g = 0; g < A.groups; ++g) {
    const X o = lane_value(worth, g);
    rank += o > worth || (o == worth && g < lane);
  }
  return __ballot(lane < A.groups && rank < A.kept);
}

// Whether this lane's i-th expert is in a group kept
template <int V>
__device__ __forceinline__ bool in_kept(unsigned long long keep, const FwdArgs& A, int lane, int i) {
  const int g = A.lanes_log2 >= 0 ? lane >> A.lanes_log2
                                  : (int)(((uint32_t)(lane * V + i) * A.magic) >> 20);
  return (keep >> (g & 63)) & 1;
}

// The choice in 64 bits: lane j gets the j-th expert.
template <int V, bool SIGMOID>
__device__ __forceinline__ int choose_wide(const FwdArgs& A, const float (&l)[V], float top, int lane,
                                           double* cs) {
  const double NEG = -__builtin_huge_val();
  double c[V], sum = 0.0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (SIGMOID) {
      c[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
      c[i] = l[i] > LOWEST ? exp((double)l[i] - (double)top) : 0.0;
      sum += c[i];
    }
  }
  if constexpr (!SIGMOID) {
    sum = wave_sum(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] *= inv;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (A.bias && lane * V + i < A.E) c[i] += (double)A.bias[lane * V + i];
    if (!(l[i] > LOWEST)) c[i] = NEG;
  }
  if (A.groups > 1) {
    const unsigned long long keep = keep_groups(group_worth<double, V>(c, A, lane, cs), A, lane);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!in_kept<V>(keep, A, lane, i)) c[i] = NEG;
  }
  if (!A.bias)  // the order of the scores is the logits'
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = c[i] > NEG ? (double)l[i] : NEG;
  int my_e = -1;
  for (int j = 0; j < A.K; ++j) {
    double head = c[0];
#pragma unroll
    for (int i = 1; i < V; ++i) head = fmax(head, c[i]);
    const double m = wave_max(head);
    if (!(m > NEG)) break;
    const int win = __ffsll((unsigned long long)__ballot(head == m)) - 1;
    int at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if ((__ballot(c[i] == m) >> win) & 1) at = i;
    const int e = win * V + at;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i == e) c[i] = NEG;
    if (lane == j) my_e = e;
  }
  return my_e;
}

// The same as a call: its registers are not the caller's
template <int V, bool SIGMOID>
__device__ __attribute__((noinline)) int choose_wide_apart(const FwdArgs& A, const float (&l)[V], float top,
                                                           int lane, double* cs) {
  return choose_wide<V, SIGMOID>(A, l, top, lane, cs);
}

// e^x by the hardware's 2^x: off by |x| 2^-23 relative at most (the rounded
// argument), a unit in the last place more
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

// How far apart two keys c = s + bias must be for their order to be sure,
// before 2^-22 |c| for the sums' own roundings.
//   sigmoid: the argument's rounding, the hardware's 2^x and reciprocal leave
//     s off by s (1 - s) (1.5 |l| + 2) 2^-24 + 3 s 2^-24 < 2^-22
//   softmax: the exponential off by (1.5 |x| + 2) 2^-24 with e^-|x| |x| < 0.4,
//     the sum of E <= 1024 terms and the quotient: < 2^-19 of the largest s
// and twice that separates two of them, twice again to be on the safe side.
template <bool SIGMOID>
__device__ __forceinline__ float key_slack(float largest) {
  return SIGMOID ? 0x1p-20f : 0x1p-17f * largest;
}
// whether the order of two keys, `below` at most `key`, is not sure
__device__ __forceinline__ bool too_close(uint32_t key, uint32_t below, float slack) {
  const float m = from_key(key), n = from_key(below);
  return below != 0 && !(m - n > slack + 0x1p-22f * fabsf(m));
}

// The first K + 1 experts of a token in the order of 64-bit sigmoid scores:
// lane j of its lanes (from lane `base` on) holds the j-th by 32-bit keys, -1
// where there is none, the order of the keys being sure but among neighbours.
template <typename T>
__device__ __forceinline__ int settle(const FwdArgs& A, const T* row, int e, int base, int lane) {
  double c = -__builtin_huge_val();
  if (e >= 0) {
    float x;
    if constexpr (sizeof(T) == 2) x = bf16_to_f32(row[e]); else x = row[e];
    c = 1.0 / (1.0 + exp(-(double)fminf(x, LARGEST))) + (double)A.bias[e];
  }
  int rank = 0;
  for (int j = 0; j <= A.K; ++j) {
    const double o = __shfl(c, base + j, 64);
    const int f = __shfl(e, base + j, 64);
    rank += o > c || (o == c && f < e);
  }
  // the other lanes keep their places
  const int to = e >= 0 ? base + rank : lane;
  return __builtin_amdgcn_ds_permute(to * 4, e);
}

// How far a group's worth may be off: a score, or half of two, by a quarter of
// the slack, and by 2^-24 of its terms' magnitude for the rounding of the terms
// c and as much for that of their sum; all that twice to be on the safe side.
__device__ __forceinline__ float worth_slack(float slack, float terms) {
  return 0.5f * slack + 0x1p-22f * terms;
}

// One wavefront a token.  Choices are to be those of 64-bit arithmetic, made
// in 32 bits: without a bias the experts' order is the logits' own, exact.
// With one, the order of the first k + 1 keys is right if neighbours differ
// by more than the slack, and the groups kept are if each is worth more than
// every one left out by what both may be off.  Where neighbours do not
// (one token in a thousand at 256 experts), settle orders the k + 1 by their
// sigmoids in 64 bits; where that is not enough (groups, the next after those,
// softmax scores, whose sum takes every expert) the token is done again in 64
// bits.  1024 tokens, top 8 of 256 in groups with a bias, some of them close:
// 6.3 us so, 8.5 with every one done again.
// Few tokens wait for one another's steps (8 tokens of 256 experts, top 8:
// 5.2 us with the launch); many are bound by instruction issue: the k maxima
// take about 25 vector instructions each at V = 4, the scores 15 for each of
// a lane's experts.
template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(NT) void fwd_kernel(FwdArgs A) {
  extern __shared__ double sh[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* logits = reinterpret_cast<const T*>(A.logits);
  const float NEG = -__builtin_huge_valf();
  double* cs = sh + (size_t)wave * A.E;
  float* scores = reinterpret_cast<float*>(cs);
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    bias[i] = A.bias && lane * V + i < A.E ? A.bias[lane * V + i] : 0.f;
  const int64_t stride = (int64_t)gridDim.x * WAVES;
  int64_t t = (int64_t)blockIdx.x * WAVES + wave;
  float l[V];
  load_row<T, V>(logits + t * A.E, A.E, lane, t < A.N, l);
  for (; t < A.N; t += stride) {
    float ahead[V];
    if (t + stride < A.N) load_row<T, V>(logits + (t + stride) * A.E, A.E, lane, true, ahead);
    float s[V];
    float top = 0.f, largest = 1.f;  // of the logits; of the scores
    if constexpr (SIGMOID) {
      // (the exponential of an absent expert is infinite: score 0)
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __builtin_amdgcn_rcpf(1.f + fast_exp(-l[i]));
    } else {
      top = l[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = wave_max(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > LOWEST ? fast_exp(l[i] - top) : 0.f;
        sum += s[i];
      }
      sum = wave_sum(sum);
      largest = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= largest;
    }
    uint32_t key[V];
    bool close = false;  // too close for 32 bits
    const float slack = key_slack<SIGMOID>(largest);
    if (A.groups > 1) {
      float c[V];
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = l[i] > LOWEST ? s[i] + bias[i] : NEG;
      float terms;
      const float worth = group_worth<float, V>(c, A, lane, scores, &terms);
      const unsigned long long keep = keep_groups(worth, A, lane);
      const bool mine = (keep >> lane) & 1;
      const float off = worth_slack(slack, terms);
      const float last = -wave_max(mine ? off - worth : NEG);
      const float next = wave_max(lane < A.groups && !mine ? worth + off : NEG);
      close = next > NEG && !(last > next);
#pragma unroll
      for (int i = 0; i < V; ++i)
        key[i] = c[i] > NEG && in_kept<V>(keep, A, lane, i) ? to_key(A.bias ? c[i] : l[i]) : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        key[i] = l[i] > LOWEST ? to_key(A.bias ? s[i] + bias[i] : l[i]) : 0u;
    }
    // for the chosen ones' lanes to read
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane * V + i < A.E) scores[lane * V + i] = s[i];
    wave_lds_sync();
    int my_e = -1;
    uint32_t my_key = 0;
    const int rounds = A.K + (A.bias ? 1 : 0);
    for (int j = 0; j < rounds; ++j) {
      uint32_t head = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) head = max(head, key[i]);
      const uint32_t m = wave_max(head);
      if (m == 0) break;
      const int win = __ffsll((unsigned long long)__ballot(head == m)) - 1;
      int at = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if ((__ballot(key[i] == m) >> win) & 1) at = i;
      const int e = win * V + at;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i == e) key[i] = 0;
      if (lane == j) {
        my_e = e;
        my_key = m;
      }
    }
    if (A.bias) {
      // lane j's key against lane j + 1's
      const uint32_t below = (uint32_t)__shfl_down((int)my_key, 1, 64);
      const unsigned long long tight = __ballot(lane < A.K && too_close(my_key, below, slack));
      if constexpr (SIGMOID) {
        if (tight != 0 && !close) {
          if ((tight >> (A.K - 1)) & 1) {  // is the first left out sure to be ahead of the next?
            uint32_t head = key[0];
#pragma unroll
            for (int i = 1; i < V; ++i) head = max(head, key[i]);
            close = too_close(key_of_lane(my_key, A.K), wave_max(head), slack);
          }
          if (!close) my_e = settle<T>(A, logits + t * A.E, my_e, 0, lane);
        }
      } else {
        close = close || tight != 0;
      }
    }
    if (lane >= A.K) my_e = -1;
    float my_s = my_e >= 0 ? scores[my_e] : 0.f;
    wave_lds_sync();
    if (close) {
      my_e = choose_wide<V, SIGMOID>(A, l, top, lane, cs);
      my_s = 0.f;
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane * V + i < A.E) scores[lane * V + i] = s[i];
      wave_lds_sync();
      if (my_e >= 0) my_s = scores[my_e];
      wave_lds_sync();
    }
    if (A.renorm) my_s /= wave_sum(my_s) + 1e-20f;  // lanes past K hold zeros
    if (lane < A.K) {
      A.expert[t * A.K + lane] = my_e;
      A.weight[t * A.K + lane] = my_s * A.scale;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = ahead[i];
  }
}

// Many tokens: several to a wavefront, L = 16 or 32 lanes each, so that the
// moves within 16 lanes serve four maxima at once.  V experts a lane, E <= L V,
// K <= 15, groups of whole lanes only.  32 lanes serve more than 256 experts
// (at 256, 65536 tokens take 51 us with 16 lanes, 59 with 32).  16384 tokens,
// top 2 of 64: 4.5 us; 8191, top 8 of 256 in groups: 14.3 us (two wavefronts a
// SIMD, waiting for the dependent steps of the rounds).  The choice in 64 bits
// is a call: inlined, its registers cost the rest (65536 tokens, top 8 of 256:
// 49 us so, 59).
template <typename X, typename F>
__device__ __forceinline__ X row_all(X x, F&& f) {
  x = f(x, other<0>(x));
  x = f(x, other<1>(x));
  x = f(x, other<2>(x));
  return f(x, other<3>(x));
}
// this lane's value and the one 16 lanes on or back, the lower lane's first
__device__ __forceinline__ void pair16(uint32_t x, uint32_t& lower, uint32_t& upper) {
  const auto v = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  lower = v[0];
  upper = v[1];
}
__device__ __forceinline__ void pair16(float x, float& lower, float& upper) {
  uint32_t a, b;
  pair16(__float_as_uint(x), a, b);
  lower = __uint_as_float(a);
  upper = __uint_as_float(b);
}
// over the lanes of a token
template <int L, typename F>
__device__ __forceinline__ float token_all(float x, F&& f) {
  x = row_all(x, f);
  if constexpr (L == 32) {
    float a, b;
    pair16(x, a, b);
    x = f(a, b);
  }
  return x;
}
// rank of this lane's group among its token's: groups of 2^LOG lanes, compared
// with those N groups on in 16 lanes, from N = 1 for its own, 0 for the others
template <int LOG, int N>
__device__ __forceinline__ int row_rank(float worth, int lane, float theirs, int from) {
  if constexpr ((N << LOG) >= 16) {
    return 0;
  } else {
    float o = theirs;
    int f = from;
    if constexpr (N > 0) {
      constexpr int CTRL = 0x120 + (N << LOG);  // row_ror
      o = dpp<CTRL>(theirs);
      f = __builtin_amdgcn_update_dpp(0, from, CTRL, 0xf, 0xf, true);
    }
    return (o > worth || (o == worth && f < lane)) + row_rank<LOG, N + 1>(worth, lane, theirs, from);
  }
}
template <int LOG, int L>
__device__ __forceinline__ int group_rank(float worth, int lane) {
  int rank = row_rank<LOG, 1>(worth, lane, worth, lane);
  if constexpr (L == 32) {
    float a, b;
    pair16(worth, a, b);
    rank += row_rank<LOG, 0>(worth, lane, lane & 16 ? a : b, lane ^ 16);
  }
  return rank;
}

template <typename T, int V, bool SIGMOID, int L>
// (four wavefronts a SIMD: 65536 tokens of 384 experts 72 us so, 90 with the
// registers of three; of 256 experts in groups 48 and 58)
__global__ __launch_bounds__(NT, V == 16 ? 4 : 1) void fwd_rows_kernel(FwdArgs A) {
  constexpr int V64 = V * L < 64 ? 1 : V * L / 64, TOKENS = 64 / L;  // of a wavefront
  constexpr int ROW = L * V + 16;  // scores, chosen
  constexpr bool APART = V * L < 64;  // the 64-bit choice's shared memory
  __shared__ alignas(16) float lds[WAVES * TOKENS * ROW + (APART ? WAVES * 128 : 0)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & (L - 1), q = lane / L;
  const T* logits = reinterpret_cast<const T*>(A.logits);
  const float NEG = -__builtin_huge_valf();
  float* scores = lds + (wave * TOKENS + q) * ROW;
  int* chosen = reinterpret_cast<int*>(scores + L * V);
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) bias[i] = A.bias && r * V + i < A.E ? A.bias[r * V + i] : 0.f;
  const int64_t stride = (int64_t)gridDim.x * WAVES * TOKENS;
  int64_t t = ((int64_t)blockIdx.x * WAVES + wave) * TOKENS + q;
  float l[V];
  load_row<T, V>(logits + t * A.E, A.E, r, t < A.N, l);
  for (; t - q < A.N; t += stride) {
    float ahead[V];
    if (t - q + stride < A.N)
      load_row<T, V>(logits + (t + stride) * A.E, A.E, r, t + stride < A.N, ahead);
    float s[V];
    float top = 0.f, largest = 1.f;
    auto fmaxf_ = [](float a, float b) { return fmaxf(a, b); };
    if constexpr (SIGMOID) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __builtin_amdgcn_rcpf(1.f + fast_exp(-l[i]));
    } else {
      top = l[0];
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = token_all<L>(top, fmaxf_);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > LOWEST ? fast_exp(l[i] - top) : 0.f;
        sum += s[i];
      }
      sum = token_all<L>(sum, [](float a, float b) { return a + b; });
      largest = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= largest;
    }
#pragma unroll
    for (int i = 0; i < V; i += V < 4 ? V : 4) {
      if constexpr (V >= 4)
        *reinterpret_cast<float4*>(scores + r * V + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      else
#pragma unroll
        for (int j = 0; j < V; ++j) scores[r * V + j] = s[j];
    }
    uint32_t key[V];
    bool close = false;
    const float slack = key_slack<SIGMOID>(largest);
    bool kept = true;
    if (A.groups > 1) {
      float b1 = NEG, b2 = NEG;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float c = l[i] > LOWEST ? s[i] + bias[i] : NEG;
        b2 = fmaxf(b2, fminf(b1, c));
        b1 = fmaxf(b1, c);
      }
      if (A.lanes_log2 > 0) merge_best<0>(b1, b2);
      if (A.lanes_log2 > 1) merge_best<1>(b1, b2);
      if (A.lanes_log2 > 2) merge_best<2>(b1, b2);
      if constexpr (L == 32)
        if (A.lanes_log2 > 3) merge_best<3>(b1, b2);
      const float worth = worth_of(b1, b2, A.best);
      const int rank = A.lanes_log2 == 0   ? group_rank<0, L>(worth, r)
                       : A.lanes_log2 == 1 ? group_rank<1, L>(worth, r)
                       : A.lanes_log2 == 2 ? group_rank<2, L>(worth, r)
                       : A.lanes_log2 == 3 ? group_rank<3, L>(worth, r)
                                           : group_rank<4, L>(worth, r);
      kept = rank < A.kept;
      const float off = worth_slack(slack, terms_of(b1, b2, A.best));
      const float last = -token_all<L>(kept ? off - worth : NEG, fmaxf_);
      const float next = token_all<L>(kept ? NEG : worth + off, fmaxf_);
      close = next > NEG && !(last > next);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      key[i] = kept && l[i] > LOWEST ? to_key(A.bias ? s[i] + bias[i] : l[i]) : 0u;
    uint32_t my_key = 0;
    const int rounds = A.K + (A.bias ? 1 : 0);
    for (int j = 0; j < rounds; ++j) {
      uint32_t head = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) head = max(head, key[i]);
      uint32_t m = max_with<0xB1>(head);
      m = max_with<0x4E>(m);
      m = max_with<0x141>(m);
      m = max_with<0x140>(m);
      if constexpr (L == 32) {
        uint32_t a, b;
        pair16(m, a, b);
        m = max(a, b);
      }
      // the lowest of the token's lanes that hold it, and there the lowest i
      const uint32_t holders = (uint32_t)(__ballot(head == m) >> (lane & (64 - L))) & (uint32_t)((1ull << L) - 1);
      bool mine = m != 0 && r == __ffs((int)holders) - 1;
      int at = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool hit = mine && key[i] == m;
        key[i] = hit ? 0u : key[i];
        at = hit ? i : at;
        mine = mine && !hit;
      }
      if (m != 0 && r == __ffs((int)holders) - 1) chosen[j] = r * V + at;
      my_key = r == j ? m : my_key;
    }
    wave_lds_sync();
    int my_e = r < rounds && my_key != 0 ? chosen[r] : -1;
    if (A.bias) {
      const uint32_t below = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)my_key, 0x101, 0xf, 0xf, true);
      const unsigned long long tight = __ballot(r < A.K && too_close(my_key, below, slack));
      if constexpr (SIGMOID) {
        if (tight != 0) {
          if ((tight >> (lane & (64 - L)) >> (A.K - 1)) & 1) {  // of this token
            // is the first left out sure to be ahead of the next?
            const uint32_t first_out = (uint32_t)__shfl((int)my_key, (lane & (64 - L)) + A.K, 64);
#pragma unroll
            for (int i = 0; i < V; ++i) close = close || too_close(first_out, key[i], slack);
          }
          // (tokens that were sure keep their order)
          my_e = settle<T>(A, logits + t * A.E, my_e, lane & (64 - L), lane);
        }
      } else {
        close = close || ((tight >> lane) & 1);
      }
    }
    if (r >= A.K) my_e = -1;
    float my_s = my_e >= 0 ? scores[my_e] : 0.f;
    wave_lds_sync();
    const unsigned long long redo = __ballot(close);
    if (redo) {
      FwdArgs W = A;
      W.lanes_log2 = A.wide_log2;
      double* cs = reinterpret_cast<double*>(lds + wave * TOKENS * ROW);
      if constexpr (APART) cs = reinterpret_cast<double*>(lds + WAVES * TOKENS * ROW + wave * 128);
      for (int k = 0; k < TOKENS; ++k) {
        if (!((redo >> (L * k)) & ((1ull << L) - 1))) continue;
        const int64_t tk = t - q + k;
        float w[V64];
        load_row<T, V64>(logits + tk * A.E, A.E, lane, tk < A.N, w);
        const float tw = __shfl(top, L * k, 64);
        const int e = __shfl(choose_wide_apart<V64, SIGMOID>(W, w, tw, lane, cs), r, 64);
        if (q == k) {
          my_e = r < A.K ? e : -1;
          my_s = 0.f;
          if (my_e >= 0) {
            float x;
            if constexpr (sizeof(T) == 2) x = bf16_to_f32(logits[t * A.E + my_e]);
            else x = logits[t * A.E + my_e];
            x = fminf(x, LARGEST);
            my_s = SIGMOID ? __builtin_amdgcn_rcpf(1.f + fast_exp(-x)) : fast_exp(x - top) * largest;
          }
        }
        wave_lds_sync();
      }
    }
    if (A.renorm) my_s /= token_all<L>(my_s, [](float a, float b) { return a + b; }) + 1e-20f;
    if (r < A.K && t < A.N) {
      A.expert[t * A.K + r] = my_e;
      A.weight[t * A.K + r] = my_s * A.scale;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = ahead[i];
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

// A sigmoid and its derivative from e = exp(-|l|) <= 1: s (1 - s) is e / (1 + e)^2
// on either side of 0, with nothing subtracted (1 - s has no bits left for a
// large l).
__device__ __forceinline__ float sigmoid_of(float l) {
  return 1.f / (1.f + expf(-l));
}
__device__ __forceinline__ float sigmoid_slope(float l) {
  const float e = expf(-fabsf(l)), d = 1.f + e;
  return e / (d * d);
}

// t_j = scale dw_j; renorm: ds_j = (t_j - sum_i t_i w_i) / S with w = s / S and
// S = sum s + 1e-20, else ds_j = t_j; then sigmoid: dl = s (1 - s) ds, softmax:
// dl = s (ds - sum ds s).  Where one weight or score h is far above a half, its
// own difference is what the others leave of it, and is formed from them:
//   ds_h = (t_h (sum_{i not h} s_i + 1e-20) / S - sum_{i not h} t_i w_i) / S
//   dl_h = s_h (ds_h sum_{i not h} s_i - sum_{i not h} ds_i s_i)
// (a wavefront without such a token passes that by).  One wavefront a token;
// slot j is lane j's.
constexpr float ALMOST = 0.6f;  // only one can be above; below, 1 - s keeps its bits
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
    float l[V], s[V], inv = 0.f;  // inv: a softmax's largest score
    load_row<T, V>(row, A.E, lane, true, l);
    if (e < 0 || e >= A.E) e = -1;
    float up = 0.f, le = -__builtin_huge_valf();
    if (e >= 0) {
      if (!A.slot_row || (r >= 0 && r < A.R)) up = A.d_weight[r] * A.scale;
      if constexpr (sizeof(T) == 2) le = bf16_to_f32(row[e]); else le = row[e];
    }
    if (!(le > LOWEST)) le = -__builtin_huge_valf();
    le = fminf(le, LARGEST);
    float se;
    if constexpr (SIGMOID) {  // s: the derivative
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = l[i] > LOWEST ? sigmoid_slope(l[i]) : 0.f;
      se = le > LOWEST ? sigmoid_of(le) : 0.f;
    } else {
      float top = l[0], sum = 0.f;
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = wave_max(top);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > LOWEST ? expf(l[i] - top) : 0.f;
        sum += s[i];
      }
      sum = wave_sum(sum);
      inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
      se = le > LOWEST ? expf(le - top) * inv : 0.f;
    }
    float d = up;
    if (A.renorm) {
      const float S = wave_sum(se) + 1e-20f, w = se / S;
      d = up - wave_sum(up * w);
      if (__ballot(w > ALMOST)) {
        const float left = wave_sum(w > ALMOST ? 0.f : se) + 1e-20f;
        const float others = wave_sum(w > ALMOST ? 0.f : up * w);
        if (w > ALMOST) d = up * (left / S) - others;
      }
      d /= S;
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
    if constexpr (!SIGMOID) {
      const float dot = wave_sum(d * se);
      if (__ballot(inv > ALMOST)) {
        float rest = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) rest += s[i] > ALMOST ? 0.f : s[i];
        rest = wave_sum(rest);
        const float others = wave_sum(se > ALMOST ? 0.f : d * se);
#pragma unroll
        for (int i = 0; i < V; ++i) ds[i] = s[i] > ALMOST ? ds[i] * rest - others : ds[i] - dot;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) ds[i] -= dot;
      }
    }
    T* out = reinterpret_cast<T*>(A.dlogits) + t * A.E;
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] *= s[i];
    store_row<T, V>(out, A.E, lane, ds);
  }
}

// Many tokens: four to a wavefront, as fwd_rows_kernel: 16384 x 64 fp32 4.0 us
// (6.1 with one), 8192 x 256 bf16 top 8 5.8 (7.4).  The slots' gradients
// meet the experts through shared memory: every slot of an expert writes the
// same sum over the expert's slots, taken in slot order.  K <= 16.
template <int J>
__device__ __forceinline__ float slot_sum(float all, int e, float d, int K) {
  if constexpr (J == 16) {
    return all;
  } else {
    if (J >= K) return all;
    constexpr int CTRL = 0x150 + J;  // row_newbcast: lane J of each row
    const int ej = __builtin_amdgcn_update_dpp(0, e, CTRL, 0xf, 0xf, true);
    const float dj = dpp<CTRL>(d);
    return slot_sum<J + 1>(all + (ej == e ? dj : 0.f), e, d, K);
  }
}

template <typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(NT) void bwd_rows_kernel(BwdArgs A) {
  __shared__ alignas(16) float lds[WAVES * 4 * 16 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
  float* mine = lds + (wave * 4 + q) * 16 * V;
  const int64_t stride = (int64_t)gridDim.x * WAVES * 4;
  for (int64_t t = ((int64_t)blockIdx.x * WAVES + wave) * 4 + q; t - q < A.N; t += stride) {
    const bool live = t < A.N;
    const T* row = reinterpret_cast<const T*>(A.logits) + t * A.E;
    int e = -1;
    int64_t at = -1;
    if (live && r < A.K) {
      e = A.expert[t * A.K + r];
      at = A.slot_row ? (int64_t)A.slot_row[t * A.K + r] : t * A.K + r;
    }
    float l[V], s[V], inv = 0.f;
    load_row<T, V>(row, A.E, r, live, l);
    if (e < 0 || e >= A.E) e = -1;
    float up = 0.f, le = -__builtin_huge_valf();
    if (e >= 0) {
      if (!A.slot_row || (at >= 0 && at < A.R)) up = A.d_weight[at] * A.scale;
      if constexpr (sizeof(T) == 2) le = bf16_to_f32(row[e]); else le = row[e];
    }
    if (!(le > LOWEST)) le = -__builtin_huge_valf();
    le = fminf(le, LARGEST);
#pragma unroll
    for (int i = 0; i < V; i += V < 4 ? V : 4) {
      if constexpr (V >= 4)
        *reinterpret_cast<float4*>(mine + r * V + i) = make_float4(0.f, 0.f, 0.f, 0.f);
      else
#pragma unroll
        for (int j = 0; j < V; ++j) mine[r * V + j] = 0.f;
    }
    auto sum_ = [](float a, float b) { return a + b; };
    float se;
    if constexpr (SIGMOID) {  // s: the derivative
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = l[i] > LOWEST ? sigmoid_slope(l[i]) : 0.f;
      se = le > LOWEST ? sigmoid_of(le) : 0.f;
    } else {
      float top = l[0], sum = 0.f;
#pragma unroll
      for (int i = 1; i < V; ++i) top = fmaxf(top, l[i]);
      top = row_all(top, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] > LOWEST ? expf(l[i] - top) : 0.f;
        sum += s[i];
      }
      sum = row_all(sum, sum_);
      inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
      se = le > LOWEST ? expf(le - top) * inv : 0.f;
    }
    float d = up;
    if (A.renorm) {
      const float S = row_all(se, sum_) + 1e-20f, w = se / S;
      d = up - row_all(up * w, sum_);
      if (__ballot(w > ALMOST)) {
        const float left = row_all(w > ALMOST ? 0.f : se, sum_) + 1e-20f;
        const float others = row_all(w > ALMOST ? 0.f : up * w, sum_);
        if (w > ALMOST) d = up * (left / S) - others;
      }
      d /= S;
    }
    if (e < 0) d = 0.f;
    const float all = slot_sum<0>(0.f, e, d, A.K);
    wave_lds_sync();
    if (e >= 0) mine[e] = all;
    wave_lds_sync();
    float ds[V];
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] = mine[r * V + i];
    wave_lds_sync();
    if constexpr (!SIGMOID) {
      const float dot = row_all(d * se, sum_);
      if (__ballot(inv > ALMOST)) {
        float rest = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) rest += s[i] > ALMOST ? 0.f : s[i];
        rest = row_all(rest, sum_);
        const float others = row_all(se > ALMOST ? 0.f : d * se, sum_);
#pragma unroll
        for (int i = 0; i < V; ++i) ds[i] = s[i] > ALMOST ? ds[i] * rest - others : ds[i] - dot;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) ds[i] -= dot;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) ds[i] *= s[i];
    if (live) store_row<T, V>(reinterpret_cast<T*>(A.dlogits) + t * A.E, A.E, r, ds);
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
constexpr int FEW = 128;

__device__ __forceinline__ int local_expert(const TablesArgs& A, int64_t f, int64_t f1) {
  if (f >= f1) return -1;
  const int32_t x = A.expert[f];
  return x >= A.first && x - A.first < A.n_local ? x - A.first : -1;
}

template <int RUN>
__global__ __launch_bounds__(RUN) void count_kernel(TablesArgs A, int pairs) {
  extern __shared__ int hist[];
  const int width = A.n_local + 1;
  const int64_t f0 = (int64_t)blockIdx.x * pairs, f1 = min(f0 + pairs, A.N * A.K);
  const int e = threadIdx.x < pairs ? local_expert(A, f0 + threadIdx.x, f1) : -1;
  for (int i = threadIdx.x; i < width; i += RUN) hist[i] = 0;
  __syncthreads();
  if (e >= 0) atomicAdd(&hist[e], 1);
  const unsigned long long on = __ballot(e >= 0);
  if ((threadIdx.x & 63) == 0) atomicAdd(&hist[A.n_local], (int)__popcll(on));
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += RUN) A.ws[(int64_t)blockIdx.x * width + i] = hist[i];
}

// 64 columns a workgroup, 16 shares of the runs, eight counts on their way at
// a time
__global__ __launch_bounds__(1024) void scan_kernel(TablesArgs A, int runs) {
  constexpr int AT_ONCE = 8;
  __shared__ int part[16][64];
  const int width = A.n_local + 1;
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int each = (runs + 15) / 16, r0 = min(share * each, runs), r1 = min(r0 + each, runs);
  int v[AT_ONCE];
  auto load = [&](int r) {
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) v[i] = r + i < r1 ? A.ws[(int64_t)(r + i) * width + e] : 0;
  };
  int sum = 0;
  if (e < width)
    for (int r = r0; r < r1; r += AT_ONCE) {
      load(r);
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) sum += v[i];
    }
  part[share][lane] = sum;
  __syncthreads();
  int base = 0;
  for (int i = 0; i < share; ++i) base += part[i][lane];
  if (e >= width) return;
  for (int r = r0; r < r1; r += AT_ONCE) {
    load(r);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      if (r + i < r1) A.ws[(int64_t)(r + i) * width + e] = base;
      base += v[i];
    }
  }
  if (share == 15) A.ws[(int64_t)runs * width + e] = base;
}

// Shares in which a workgroup of place_kernel adds up the other runs' counts,
// one thread for each share of an expert.  At most 16, which one thread adds
// up in turn: 32768 pairs of one local expert 6.9 us so, 9.3 without a limit,
// 7.5 and 8.7 with 8 and 4.
__host__ __device__ __forceinline__ int shares_of(int run, int width) {
  const int s = run / width;
  return s < 1 ? 1 : s > 16 ? 16 : s;
}

// shared memory of place_kernel, in ints
template <int RUN>
static size_t place_lds(int n_local) {
  const size_t width = (size_t)n_local + 1;
  const size_t shares = shares_of(RUN, (int)width);
  return 2 * width + RUN + RUN / 64 * 2 + 2 * shares * width + ((size_t)RUN / 64 * n_local + 1) / 2;
}

template <int RUN>
__global__ __launch_bounds__(RUN) void place_kernel(TablesArgs A, int pairs, int runs) {
  constexpr int WV = RUN / 64;
  extern __shared__ int lds[];
  const int width = A.n_local + 1;
  const int shares = shares_of(RUN, width);
  int* first = lds;            // [width] first row of each expert in this run
  int* total = first + width;  // [width] rows of each expert in all
  int* seen = total + width;   // [RUN] experts of this run's pairs
  int* red = seen + RUN;       // [2 WV]
  int* sums = red + 2 * WV;    // [2][shares][width] other runs' counts: earlier, all
  uint16_t* waves = reinterpret_cast<uint16_t*>(sums + 2 * shares * width);  // [WV][n_local]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int run = blockIdx.x;
  const int64_t f0 = (int64_t)run * pairs, f1 = min(f0 + pairs, A.N * A.K), f = f0 + tid;
  const int e = tid < pairs ? local_expert(A, f, f1) : -1;
  // the other runs' counts, column by column
  if (runs > FEW) {
    for (int i = tid; i < width; i += RUN) {
      sums[i] = A.ws[(int64_t)run * width + i];
      sums[width + i] = A.ws[(int64_t)runs * width + i];
    }
  } else if (runs > 1) {
    // counts on their way at a time (65528 pairs of 256 local experts 12.7 us
    // so, 14.4 with eight, 18.3 with four)
    constexpr int AT_ONCE = 16;
    for (int i = tid; i < width * shares; i += RUN) {
      const int share = i / width, col = i - share * width;
      int before = 0, all = 0;
      int r = share;
      auto batch = [&](auto whole) {
        int v[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
          v[j] = whole || r + j * shares < runs ? A.ws[(r + j * shares) * width + col] : 0;
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
          all += v[j];
          before += r + j * shares < run ? v[j] : 0;
        }
      };
      for (; r + (AT_ONCE - 1) * shares < runs; r += AT_ONCE * shares) batch(std::true_type{});
      if (r < runs) batch(std::false_type{});
      sums[i] = before;
      sums[shares * width + i] = all;
    }
  }
  const int parts = runs > FEW ? 1 : shares;
  seen[tid] = e;
  // rank among the lanes with the same expert
  const unsigned long long below = (1ull << lane) - 1;
  const unsigned long long on = __ballot(e >= 0);
  unsigned long long same = on;
  for (int b = 0; (1 << b) < A.n_local; ++b) {
    const unsigned long long bit = __ballot((e >> b) & 1);
    same &= (e >> b) & 1 ? bit : ~bit;
  }
  const int rank = __popcll(same & below);
  uint16_t* mine = waves + wave * A.n_local;
  for (int i = lane; i < A.n_local; i += 64) mine[i] = 0;
  wave_lds_sync();
  if (e >= 0 && rank == 0) mine[e] = (uint16_t)__popcll(same);
  if (lane == 0) red[wave] = __popcll(on);
  __syncthreads();
  // each expert's pairs in earlier wavefronts, in earlier runs and in all
  int all = 0, before = 0;
  if (tid < A.n_local) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < WV; ++w) {
      const int v = waves[w * A.n_local + tid];
      waves[w * A.n_local + tid] = (uint16_t)sum;
      sum += v;
    }
    all = sum;
  }
  if (runs > 1 && tid < width) {
    all = 0;
    for (int p = 0; p < parts; ++p) {
      before += sums[p * width + tid];
      all += sums[(parts + p) * width + tid];
    }
  }
  int earlier_waves = 0, listed = 0;  // list entries in earlier wavefronts, and of the run
#pragma unroll
  for (int w = 0; w < WV; ++w) {
    const int v = red[w];
    earlier_waves += w < wave ? v : 0;
    listed += v;
  }
  // an expert's first row: the totals of the experts before it, chunks of
  // RUN experts (one where n_local fits the workgroup)
  int carry = 0;
  for (int e0 = 0; e0 < A.n_local; e0 += RUN) {
    if (e0 > 0) {  // n_local > RUN: this thread's next expert
      const int i = e0 + tid;
      all = before = 0;
      if (i < A.n_local) {
        int sum = 0;
        for (int w = 0; w < WV; ++w) {
          const int v = waves[w * A.n_local + i];
          waves[w * A.n_local + i] = (uint16_t)sum;
          sum += v;
        }
        all = sum;
        if (runs > 1) {
          all = 0;
          for (int p = 0; p < parts; ++p) {
            before += sums[p * width + i];
            all += sums[(parts + p) * width + i];
          }
        }
      }
    }
    const int v = e0 + tid < A.n_local ? all : 0;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(x, d, 64);
      if (lane >= d) x += u;
    }
    int base = carry + x - v;
    if (A.n_local > 64) {
      __syncthreads();
      if (lane == 63) red[WV + wave] = x;
      __syncthreads();
      for (int w = 0; w < wave; ++w) base += red[WV + w];
      for (int w = 0; w < WV; ++w) carry += red[WV + w];
    }
    if (e0 + tid < A.n_local) {
      first[e0 + tid] = base + before;
      total[e0 + tid] = all;
      if (run == 0) A.offsets[e0 + tid] = base;
    }
  }
  // the lists' own sums: column n_local
  if (tid == RUN - 1) {
    int b = 0, t = listed;
    if (runs > 1) {
      t = 0;
      for (int p = 0; p < parts; ++p) {
        b += sums[p * width + A.n_local];
        t += sums[(parts + p) * width + A.n_local];
      }
    }
    first[A.n_local] = b;
    total[A.n_local] = t;
    if (run == 0) {
      A.offsets[A.n_local] = t;
      A.tok_ptr[A.N] = t;
    }
  }
  __syncthreads();
  for (int64_t r = total[A.n_local] + (int64_t)run * RUN + tid; r < A.R; r += (int64_t)gridDim.x * RUN) {
    A.row_token[r] = -1;
    A.tok_rows[r] = -1;
    if (A.row_weight) A.row_weight[r] = 0.f;
  }
  if (tid >= pairs || f >= f1) return;
  const int token = tid / A.K, slot = tid - token * A.K;
  const int t = run * (pairs / A.K) + token;
  // list entries of this token's earlier slots, and of its lower rows
  int earlier = 0, lower = 0;
  for (int i = 0; i < A.K; ++i) {
    const int o = seen[token * A.K + i];
    if (o < 0) continue;
    earlier += i < slot;
    lower += o < e || (o == e && i < slot);
  }
  const int start = first[A.n_local] + earlier_waves + __popcll(on & below) - earlier;
  if (slot == 0) A.tok_ptr[t] = start;
  int row = -1;
  if (e >= 0) {
    row = first[e] + waves[wave * A.n_local + e] + rank;
    A.tok_rows[start + lower] = row;
    A.row_token[row] = t;
    if (A.row_weight) A.row_weight[row] = A.weight[f];
  }
  A.slot_row[f] = row;
}

// Threads of a run, a pair each: one run where that is possible (one launch),
// else the smallest runs whose counts place_kernel adds up itself (two), with
// at most 24 counts a thread.  32768 pairs: of 8 local experts 7.1 us with runs
// of 256 and 512 threads, 7.7 with 1024; of 64 (33 counts a thread, 8, 2) 8.8,
// 8.3 and 9.6; of 256 (129, 32, 8) 14.4, 10.3 and 10.9.  8192 pairs of 32 (4
// counts, 1) 7.5 and 8.0.
static int run_threads(int64_t N, int K, int n_local) {
  if (N * K > 256 && (N + 1024 / K - 1) / (1024 / K) <= 1) return 1024;
  for (int run = 256; run < 1024; run *= 2)
    if ((N + run / K - 1) / (run / K) <= FEW && N * K * (n_local + 1) <= 24 * (int64_t)run * run)
      return run;
  return 1024;
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

template <typename F>
static void pick_rows(int dtype, int V, int score, F&& f) {
  auto by_score = [&](auto t, auto v) {
    score == TP_SCORE_SIGMOID ? f(t, v, std::true_type{}) : f(t, v, std::false_type{});
  };
  auto by_size = [&](auto t) {
    V == 1   ? by_score(t, std::integral_constant<int, 1>{})
    : V == 2 ? by_score(t, std::integral_constant<int, 2>{})
    : V == 4 ? by_score(t, std::integral_constant<int, 4>{})
    : V == 8 ? by_score(t, std::integral_constant<int, 8>{})
             : by_score(t, std::integral_constant<int, 16>{});
  };
  dtype == TP_BF16 ? by_size(bf16_t{}) : by_size(0.f);
}

// Tokens from which several of them share a wavefront: then those wavefronts
// fill the chip.  Forward, top 2 of 64: 2048 tokens 3.3 us so and 3.1 with a
// wavefront each, 4096 3.1 and 3.6, 32768 6.4 and 12.5; top 8 of 256 (16 experts
// a lane): 6144 8.1 and 7.7, 7168 8.2 and 8.8, 12288 9.6 and 14.1; top 8 of 512
// (32 lanes a token): 4096 8.0 and 10.3, 8192 11.1 and 17.4.
static int64_t rows_from(int E) { return E <= 128 || E > 256 ? 4096 : 7168; }
constexpr int64_t ROWS_GRID = 1024;
// experts of a lane with 16 lanes a token
static int rows_experts(int E) { return E <= 16 ? 1 : E <= 32 ? 2 : E <= 64 ? 4 : E <= 128 ? 8 : 16; }

static unsigned grid_tokens(int64_t N, int64_t most) {
  const int64_t b = (N + WAVES - 1) / WAVES;
  return (unsigned)(b > most ? most : b);
}

}  // namespace route

hipError_t route_fwd_launch(const tp_route_desc& d, const void* logits, const float* bias,
                            int32_t* expert, float* weight, hipStream_t st) {
  using namespace route;
  if (d.N == 0) return hipSuccess;
  const int per = d.E / d.groups;
  FwdArgs a{logits, bias, expert, weight, d.N, d.E, d.K, d.groups, d.groups_kept, d.group_best,
            d.renorm, d.scale, per, -1, (uint32_t)(((1 << 20) + per - 1) / per), -1};
  auto log2_lanes = [&](int V) {
    for (int b = 0; b <= 4; ++b)
      if (per == V << b) return b;
    return -1;
  };
  const int L = d.E <= 256 ? 16 : 32;
  const int v = L == 16 ? rows_experts(d.E) : 16;
  const int64_t from = rows_from(d.E);
  const int lanes = log2_lanes(v);
  if (d.N >= from && d.E <= v * L && d.K <= 15 && (d.groups == 1 || (lanes >= 0 && lanes <= (L == 32 ? 4 : 3)))) {
    const int tokens = WAVES * (64 / L);
    const int64_t groups = (d.N + tokens - 1) / tokens;
    const dim3 grid((unsigned)(groups > ROWS_GRID ? ROWS_GRID : groups));
    a.lanes_log2 = lanes;
    a.wide_log2 = log2_lanes(v * L < 64 ? 1 : v * L / 64);
    pick_rows(d.dtype, v, d.score, [&](auto t, auto v, auto sig) {
      constexpr int V = decltype(v)::value;
      if constexpr (V == 16) {
        if (L == 32) {
          hipLaunchKernelGGL((fwd_rows_kernel<decltype(t), V, decltype(sig)::value, 32>), grid, dim3(NT), 0,
                             st, a);
          return;
        }
      }
      hipLaunchKernelGGL((fwd_rows_kernel<decltype(t), V, decltype(sig)::value, 16>), grid, dim3(NT), 0, st, a);
    });
    return hipGetLastError();
  }
  return pick(d.dtype, d.E, d.score, [&](auto t, auto v, auto sig) {
    constexpr int V = decltype(v)::value;
    a.lanes_log2 = log2_lanes(V);
    hipLaunchKernelGGL((fwd_kernel<decltype(t), V, decltype(sig)::value>), dim3(grid_tokens(d.N, 1024)),
                       dim3(NT), (size_t)WAVES * d.E * sizeof(double), st, a);
    return hipGetLastError();
  });
}

hipError_t route_bwd_launch(const tp_route_desc& d, const void* logits, const int32_t* expert,
                            const float* d_weight, const int32_t* slot_row, int64_t R,
                            void* dlogits, hipStream_t st) {
  using namespace route;
  if (d.N == 0) return hipSuccess;
  BwdArgs a{logits, expert, d_weight, slot_row, dlogits, d.N, R, d.E, d.K, d.renorm, d.scale};
  // Where the experts are no whole lanes, single loads and stores cost more than
  // shared wavefronts give, but for few bf16 experts.  8192 tokens, bf16: of 256
  // 5.8 us so and 7.4 with a wavefront each, of 200 10.9 and 7.3, of 136 8.7 and
  // 6.8, of 100 5.2 and 5.8; fp32: of 256 7.6 and 7.8, of 200 14.6 and 7.6, of
  // 144 5.9 and 7.0, of 100 6.7 and 5.9.
  const bool whole = d.E % rows_experts(d.E) == 0;
  if (d.N >= rows_from(d.E) && d.E <= 256 && d.K <= 16 && (whole || (d.E <= 128 && d.dtype == TP_BF16))) {
    const int64_t groups = (d.N + 4 * WAVES - 1) / (4 * WAVES);
    const dim3 grid((unsigned)(groups > 2 * ROWS_GRID ? 2 * ROWS_GRID : groups));
    pick_rows(d.dtype, rows_experts(d.E), d.score, [&](auto t, auto v, auto sig) {
      hipLaunchKernelGGL((bwd_rows_kernel<decltype(t), decltype(v)::value, decltype(sig)::value>),
                         grid, dim3(NT), 0, st, a);
    });
    return hipGetLastError();
  }
  return pick(d.dtype, d.E, d.score, [&](auto t, auto v, auto sig) {
    hipLaunchKernelGGL((bwd_kernel<decltype(t), decltype(v)::value, decltype(sig)::value>),
                       dim3(grid_tokens(d.N, 8192)), dim3(NT), 0, st, a);
    return hipGetLastError();
  });
}

size_t route_tables_workspace(int64_t N, int K, int n_local) {
  const int64_t tokens = route::run_threads(N, K, n_local) / K;
  const int64_t runs = (N + tokens - 1) / tokens;
  if (runs <= 1) return 16;  // not used; a caller need not tell sizes apart
  return (size_t)(runs + (runs > route::FEW ? 1 : 0)) * ((size_t)n_local + 1) * sizeof(int32_t);
}

template <int RUN>
static hipError_t tables_launch(const TablesArgs& a, hipStream_t st) {
  using namespace route;
  const int tokens = RUN / a.K, pairs = tokens * a.K;
  const int runs = (int)((a.N + tokens - 1) / tokens);
  const size_t width = (size_t)a.n_local + 1;
  hipError_t he = hipSuccess;
  if (runs > 1) {
    hipLaunchKernelGGL(count_kernel<RUN>, dim3((unsigned)runs), dim3(RUN), width * sizeof(int), st, a,
                       pairs);
    if ((he = hipGetLastError()) != hipSuccess) return he;
  }
  if (runs > FEW) {
    hipLaunchKernelGGL(scan_kernel, dim3((unsigned)((width + 63) / 64)), dim3(1024), 0, st, a, runs);
    if ((he = hipGetLastError()) != hipSuccess) return he;
  }
  hipLaunchKernelGGL(place_kernel<RUN>, dim3((unsigned)(runs > 0 ? runs : 1)), dim3(RUN),
                     place_lds<RUN>(a.n_local) * sizeof(int), st, a, pairs, runs);
  return hipGetLastError();
}

hipError_t route_tables_launch(const TablesArgs& a, hipStream_t st) {
  switch (route::run_threads(a.N, a.K, a.n_local)) {
    case 256: return tables_launch<256>(a, st);
    case 512: return tables_launch<512>(a, st);
    default: return tables_launch<1024>(a, st);
  }
}

}  // namespace tpmlp
