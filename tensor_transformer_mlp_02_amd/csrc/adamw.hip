// AdamW over many tensors (Megatron-LM 源码精读——大模型并行训练全景 §五: fp32
// main parameters and gradients, bf16 weights).  Per element
//   m = b1 m + (1-b1) g,  v = b2 v + (1-b2) g^2,
//   p = p (1 - lr wd) - lr/c1 * m / (sqrt(v)/sqrt(c2) + eps)
// Nothing is reused: the kernel is HBM-bound at 30 bytes an element with
// fp32 states (fp32 gradient, bf16 copy) and 18 with 8-bit ones.
//
// The tensors travel by value in the kernel's arguments, up to TENSORS
// of them in a launch, so that nothing has to be copied to the device and a
// captured graph holds its own table.
#include "block_launch.h"
#include "common.h"

// Every operation below is rounded by itself: the 8-bit states' codes hang
// on the exact fp32 values, which a contraction into a multiply-add that
// the compiler may or may not make would change.
#pragma clang fp contract(off)

namespace tpmlp {
namespace adamw {

constexpr int NT = 256;
constexpr int TENSORS = 44;        // of one launch: the arguments stay under 4 KiB
// Elements of one workgroup's piece of a tensor.  fp32 states, 88M elements:
// 471 us at 4096, 472 at 2048, 489 at 8192; 8-bit, 138M: 453 us at 1024, 449 at
// 2048, 459 at 4096 (fewer wavefronts), and small tensors spread further.
constexpr int SPAN32 = 4096, SPAN8 = 1024;
// Workgroups of one launch: a grid holds fewer than 2^32 threads.
constexpr int64_t GROUPS = ((int64_t)1 << 32) / NT - 1;
constexpr int BLOCK = TP_ADAMW_BLOCK;
constexpr float FMAX = 448.f;      // largest finite E4M3

struct Tensor {
  float* p;
  bf16_t* p16;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  int64_t count;
  float wd;
};

struct Args {
  Tensor t[TENSORS];
  int first[TENSORS];  // workgroup of each one's first piece
  int n, place;  // tensors here; place of the first in the caller's list
  int64_t done;  // pieces of the first that earlier launches did
  const int32_t* dev_step;
  const float* dev_lr;
  const float* grad_scale;
  float lr, b1, b2, omb1, omb2, eps;
  float step_size, inv_root_c2;  // lr / c1 and 1 / sqrt(c2) (host step and lr)
  float inv_c1;
  float log_b1, log_b2;
  int step;
  uint32_t seed;
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

// 32 bits mixed by two multiplications with the fractions of sqrt 2 and
// sqrt 3 (odd, so that each is a bijection) between shifts
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Nothing is used again before the step has passed over everything: past
// the caches.  88M elements, fp32 states: 465 us so, 474 with plain stores,
// 487 with plain loads and stores.
typedef float f32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ float4 ld4(const float* p) {
  const f32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p));
  return make_float4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void st4(float* p, const float4& q) {
  const f32x4_t v = {q.x, q.y, q.z, q.w};
  __builtin_nontemporal_store(v, reinterpret_cast<f32x4_t*>(p));
}

struct Scalars {
  float step_size, inv_root_c2, eps, decay, gs;
  uint32_t key;
};

// this launch's scalars for tensor k; false: the step is skipped
__device__ __forceinline__ bool scalars(const Args& A, int k, Scalars& s) {
  s.gs = A.grad_scale ? *A.grad_scale : 1.f;
  if (!(fabsf(s.gs) <= 3.4028235e38f)) return false;
  const float lr = A.dev_lr ? *A.dev_lr : A.lr;
  int step = A.step;
  float inv_c1 = A.inv_c1;
  s.inv_root_c2 = A.inv_root_c2;
  if (A.dev_step) {
    step = *A.dev_step;
    if (step < 1) return false;
    // 1 - b^t = -expm1(t log b): no cancellation at small t
    inv_c1 = 1.f / -expm1f((float)step * A.log_b1);
    s.inv_root_c2 = 1.f / sqrtf(-expm1f((float)step * A.log_b2));
  }
  s.step_size = A.dev_lr || A.dev_step ? lr * inv_c1 : A.step_size;
  s.eps = A.eps;
  s.decay = 1.f - lr * A.t[k].wd;
  s.key = mix(mix(mix(A.seed) + (uint32_t)step) + (uint32_t)(A.place + k));
  return true;
}

// the last tensor whose first piece is not behind workgroup b: one look by
// all lanes
__device__ __forceinline__ int find_tensor(const Args& A, int b) {
  static_assert(TENSORS <= 64, "a lane for each");
  const int lane = threadIdx.x & 63;
  const bool before = lane < A.n && A.first[lane < TENSORS ? lane : 0] <= b;
  return __popcll(__ballot(before)) - 1;
}

// which piece of tensor k workgroup b has
__device__ __forceinline__ int64_t piece_of(const Args& A, int k, int b) {
  return b - A.first[k] + (k == 0 ? A.done : 0);
}

// four neighbours; fewer at a tensor's end
template <typename GT> struct Grad4;
template <> struct Grad4<float> {
  float4 q;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    q = ld4(reinterpret_cast<const float*>(p) + i);
  }
  __device__ __forceinline__ void get(float g[4]) const { g[0] = q.x; g[1] = q.y; g[2] = q.z; g[3] = q.w; }
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return reinterpret_cast<const float*>(p)[i];
  }
};
template <> struct Grad4<bf16_t> {
  uint2 q;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    q = *reinterpret_cast<const uint2*>(reinterpret_cast<const bf16_t*>(p) + i);
  }
  __device__ __forceinline__ void get(float g[4]) const {
    g[0] = __uint_as_float(q.x << 16);
    g[1] = __uint_as_float(q.x & 0xffff0000u);
    g[2] = __uint_as_float(q.y << 16);
    g[3] = __uint_as_float(q.y & 0xffff0000u);
  }
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return bf16_to_f32(reinterpret_cast<const bf16_t*>(p)[i]);
  }
};

__device__ __forceinline__ float new_param(float p, float m, float root, const Scalars& s) {
  return p * s.decay - s.step_size * (m / (root * s.inv_root_c2 + s.eps));
}

// fp32 states: four neighbours a thread, every load of a workgroup's piece
// before the first store
template <typename GT>
__global__ __launch_bounds__(NT) void step32_kernel(Args A) {
  const int k = find_tensor(A, blockIdx.x);
  const Tensor& t = A.t[k];
  Scalars s;
  if (!scalars(A, k, s)) return;
  const int64_t i0 = piece_of(A, k, blockIdx.x) * SPAN32;
  float* mp = reinterpret_cast<float*>(t.m);
  float* vp = reinterpret_cast<float*>(t.v);
  auto update = [&](float& p, float g, float& m, float& v) {
    g *= s.gs;
    m = m * A.b1 + g * A.omb1;
    v = v * A.b2 + g * g * A.omb2;
    p = new_param(p, m, sqrtf(v), s);
  };
  if (i0 + SPAN32 <= t.count) {
    constexpr int U = SPAN32 / (4 * NT);
    float4 p[U], m[U], v[U];
    Grad4<GT> g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + (u * NT + threadIdx.x) * 4;
      p[u] = ld4(t.p + i);
      g[u].load(t.g, i);
      m[u] = ld4(mp + i);
      v[u] = ld4(vp + i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + (u * NT + threadIdx.x) * 4;
      float gg[4];
      g[u].get(gg);
      update(p[u].x, gg[0], m[u].x, v[u].x);
      update(p[u].y, gg[1], m[u].y, v[u].y);
      update(p[u].z, gg[2], m[u].z, v[u].z);
      update(p[u].w, gg[3], m[u].w, v[u].w);
      st4(mp + i, m[u]);
      st4(vp + i, v[u]);
      st4(t.p + i, p[u]);
      if (t.p16)
        *reinterpret_cast<uint2*>(t.p16 + i) =
            make_uint2(pack_bf16x2(p[u].x, p[u].y), pack_bf16x2(p[u].z, p[u].w));
    }
    return;
  }
  // a tensor's last piece: up to three elements over, for the threads with
  // least to do, and four neighbours a thread
  const int64_t fours = t.count & ~(int64_t)3, over = fours + (NT - 1 - threadIdx.x);
  const bool one = over < t.count;
  float p1 = 0.f, g1 = 0.f, m1 = 0.f, v1 = 0.f;
  if (one) {
    p1 = t.p[over];
    g1 = Grad4<GT>::one(t.g, over);
    m1 = mp[over];
    v1 = vp[over];
  }
#pragma unroll 1
  for (int64_t i = i0 + threadIdx.x * 4; i < fours; i += NT * 4) {
    float4 p = ld4(t.p + i), m = ld4(mp + i), v = ld4(vp + i);
    Grad4<GT> g;
    g.load(t.g, i);
    float gg[4];
    g.get(gg);
    update(p.x, gg[0], m.x, v.x);
    update(p.y, gg[1], m.y, v.y);
    update(p.z, gg[2], m.z, v.z);
    update(p.w, gg[3], m.w, v.w);
    st4(mp + i, m);
    st4(vp + i, v);
    st4(t.p + i, p);
    if (t.p16)
      *reinterpret_cast<uint2*>(t.p16 + i) = make_uint2(pack_bf16x2(p.x, p.y), pack_bf16x2(p.z, p.w));
  }
  if (one) {
    update(p1, g1, m1, v1);
    mp[over] = m1;
    vp[over] = v1;
    t.p[over] = p1;
    if (t.p16) t.p16[over] = f32_to_bf16(p1);
  }
}

// the largest over the wavefront, whole: within 16 lanes by moves between
// them, then lane by lane
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max_with<0xB1>(x);   // lane ^ 1
  x = max_with<0x4E>(x);   // lane ^ 2
  x = max_with<0x141>(x);  // within 8: lane 7 - i
  x = max_with<0x140>(x);  // within 16: lane 15 - i
  auto row = [&](int i) { return (uint32_t)__builtin_amdgcn_readlane((int)x, 16 * i); };
  return max(max(row(0), row(1)), max(row(2), row(3)));
}

// Scales and their inverses of a block whose largest magnitudes have these
// bits (bits of non-negative floats order like the floats, NaN above all):
// top / 448 and 448 / top, 0 where top is at most 2^-100.  An infinity makes
// the scale NaN, like a NaN: the block's state says so.  One division serves
// all four quotients, a lane for each.
struct Scales {
  float m, m_inv, v, v_inv;
};
__device__ __forceinline__ Scales block_scales(uint32_t m, uint32_t v, int lane) {
  const float top = __uint_as_float(lane & 2 ? v : m);
  const float q = (lane & 1 ? FMAX : top) / (lane & 1 ? top : FMAX);
  auto at = [&](int i) { return __builtin_amdgcn_readlane(__float_as_int(q), i); };
  constexpr uint32_t TINY = (127u - 100u) << 23, INFINITE = 0x7f800000u;
  const int nan = 0x7fc00000;
  auto usable = [&](uint32_t bits) { return bits > TINY && bits < INFINITE; };
  return {__int_as_float(usable(m) ? at(0) : m < INFINITE ? 0 : nan),
          __int_as_float(usable(m) ? at(1) : 0),
          __int_as_float(usable(v) ? at(2) : v < INFINITE ? 0 : nan),
          __int_as_float(usable(v) ? at(3) : 0)};
}

// t rounded to an E4M3 value, down or up by a chance u = h / 2^16.  The step
// between neighbouring values at |t| in [2^k, 2^(k+1)) is 2^(k-3), and 2^-9
// below 2^-6.
//   a plain value: floor(t + u) in steps, t on average
//   a root: up from k steps with the chance (t^2 - k^2) / ((k+1)^2 - k^2),
//     so that its square, the second moment, is kept on average (a root kept
//     on average would add the rounding's variance to v at every step); a
//     positive one never becomes 0
// The variance that this adds stays small: a state that moves by d steps of
// its code is moved up or down with a chance of about d.  u and its product
// with 2 k + 1 are exact, so the multiply-adds round as the sums would.  (A
// NaN becomes some value: its block's scale is NaN.)
template <bool ROOT>
__device__ __forceinline__ float round_e4m3(float t, float h, bool positive) {
  const uint32_t power = max(__float_as_uint(t) & 0x7f800000u, (127u - 6u) << 23);  // 2^k
  t = t * __uint_as_float(((254u + 3u) << 23) - power);
  const float step = __uint_as_float(power - (3u << 23));
  if constexpr (ROOT) {
    float k = floorf(t);
    const float odd = 2.f * k + 1.f;
    k += fmaf(h, odd * 0x1p-16f, (t - k) * (t + k)) >= odd ? 1.f : 0.f;
    k = fmaxf(k, positive ? 1.f : 0.f);
    return fminf(k * step, FMAX);
  } else {
    return __builtin_amdgcn_fmed3f(floorf(fmaf(h, 0x1p-16f, t)) * step, -FMAX, FMAX);
  }
}

// 8-bit states: a wavefront takes a block of 256, four neighbours a lane,
// and requests all its blocks of a workgroup's piece at once
template <typename GT>
__global__ __launch_bounds__(NT) void step8_kernel(Args A) {
  constexpr int U = SPAN8 / (NT / 64) / BLOCK;  // blocks of a wavefront
  const int k = find_tensor(A, blockIdx.x);
  const Tensor& t = A.t[k];
  Scalars s;
  if (!scalars(A, k, s)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i0 = piece_of(A, k, blockIdx.x) * SPAN8 + wave * BLOCK;
  uint8_t* mc = reinterpret_cast<uint8_t*>(t.m);
  uint8_t* vc = reinterpret_cast<uint8_t*>(t.v);
  float4 p4[U];
  Grad4<GT> g4[U];
  uint32_t m4[U], v4[U];
  float ms[U], vs[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b0 = i0 + u * (NT / 64) * BLOCK, i = b0 + lane * 4;
    if (b0 + BLOCK > t.count) continue;
    p4[u] = ld4(t.p + i);
    g4[u].load(t.g, i);
    m4[u] = *reinterpret_cast<const uint32_t*>(mc + i);
    v4[u] = *reinterpret_cast<const uint32_t*>(vc + i);
    ms[u] = t.ms[b0 / BLOCK];
    vs[u] = t.vs[b0 / BLOCK];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b0 = i0 + u * (NT / 64) * BLOCK, i = b0 + lane * 4;
    if (b0 >= t.count) break;
    const bool whole = b0 + BLOCK <= t.count;
    const int here = whole ? 4 : (int)max((int64_t)0, min((int64_t)4, t.count - i));
    float p[4], g[4], m[4], r[4];
    float sm = ms[u], sv = vs[u];
    uint32_t cm = m4[u], cv = v4[u];
    if (whole) {
      p[0] = p4[u].x; p[1] = p4[u].y; p[2] = p4[u].z; p[3] = p4[u].w;
      g4[u].get(g);
    } else {  // a tensor's last block
      cm = cv = 0;
      sm = t.ms[b0 / BLOCK];
      sv = t.vs[b0 / BLOCK];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = g[j] = 0.f;
        if (j < here) {
          p[j] = t.p[i + j];
          g[j] = Grad4<GT>::one(t.g, i + j);
          cm |= (uint32_t)mc[i + j] << (8 * j);
          cv |= (uint32_t)vc[i + j] << (8 * j);
        }
      }
    }
    m[0] = __builtin_amdgcn_cvt_f32_fp8((int)cm, 0) * sm;
    m[1] = __builtin_amdgcn_cvt_f32_fp8((int)cm, 1) * sm;
    m[2] = __builtin_amdgcn_cvt_f32_fp8((int)cm, 2) * sm;
    m[3] = __builtin_amdgcn_cvt_f32_fp8((int)cm, 3) * sm;
    r[0] = __builtin_amdgcn_cvt_f32_fp8((int)cv, 0) * sv;
    r[1] = __builtin_amdgcn_cvt_f32_fp8((int)cv, 1) * sv;
    r[2] = __builtin_amdgcn_cvt_f32_fp8((int)cv, 2) * sv;
    r[3] = __builtin_amdgcn_cvt_f32_fp8((int)cv, 3) * sv;
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float gj = g[j] * s.gs;
      m[j] = m[j] * A.b1 + gj * A.omb1;
      r[j] = sqrtf(r[j] * r[j] * A.b2 + gj * gj * A.omb2);
      p[j] = new_param(p[j], m[j], r[j], s);
      // (past the tensor's end the states are zeros unless a scale is NaN)
      if (j < here) {
        mtop = max(mtop, __float_as_uint(m[j]) & 0x7fffffffu);
        vtop = max(vtop, __float_as_uint(r[j]) & 0x7fffffffu);
      }
    }
    const Scales sc = block_scales(wave_max(mtop), wave_max(vtop), lane);
    if (lane == 0) {
      t.ms[b0 / BLOCK] = sc.m;
      t.vs[b0 / BLOCK] = sc.v;
    }
    float km[4], kr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = mix(((uint32_t)(i + j) ^ s.key) + (uint32_t)(i >> 32));
      km[j] = round_e4m3<false>(m[j] * sc.m_inv, (float)(h & 0xffffu), false);
      kr[j] = round_e4m3<true>(r[j] * sc.v_inv, (float)(h >> 16), r[j] > 0.f);
    }
    // exact: the values are E4M3 already
    int wm = __builtin_amdgcn_cvt_pk_fp8_f32(km[0], km[1], 0, false);
    wm = __builtin_amdgcn_cvt_pk_fp8_f32(km[2], km[3], wm, true);
    int wv = __builtin_amdgcn_cvt_pk_fp8_f32(kr[0], kr[1], 0, false);
    wv = __builtin_amdgcn_cvt_pk_fp8_f32(kr[2], kr[3], wv, true);
    if (whole) {
      *reinterpret_cast<uint32_t*>(mc + i) = (uint32_t)wm;
      *reinterpret_cast<uint32_t*>(vc + i) = (uint32_t)wv;
      st4(t.p + i, make_float4(p[0], p[1], p[2], p[3]));
      if (t.p16)
        *reinterpret_cast<uint2*>(t.p16 + i) =
            make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < here) {
          mc[i + j] = (uint8_t)((uint32_t)wm >> (8 * j));
          vc[i + j] = (uint8_t)((uint32_t)wv >> (8 * j));
          t.p[i + j] = p[j];
          if (t.p16) t.p16[i + j] = f32_to_bf16(p[j]);
        }
    }
  }
}

}  // namespace adamw

hipError_t adamw_launch(const tp_adamw_desc& d, int n, const tp_adamw_tensor* t,
                        const int32_t* dev_step, const float* dev_lr, const float* grad_scale,
                        hipStream_t st) {
  using namespace adamw;
  Args a;
  a.dev_step = dev_step;
  a.dev_lr = dev_lr;
  a.grad_scale = grad_scale;
  a.lr = (float)d.lr;
  a.b1 = (float)d.beta1;
  a.b2 = (float)d.beta2;
  a.omb1 = (float)(1.0 - d.beta1);
  a.omb2 = (float)(1.0 - d.beta2);
  a.eps = (float)d.eps;
  a.step = d.step;
  a.seed = d.seed;
  // beta = 0: log is -inf and expm1 gives -1, c = 1
  a.log_b1 = (float)log(d.beta1);
  a.log_b2 = (float)log(d.beta2);
  const double c1 = 1.0 - pow(d.beta1, d.step), c2 = 1.0 - pow(d.beta2, d.step);
  a.inv_c1 = (float)(1.0 / c1);
  a.step_size = (float)(d.lr / c1);
  a.inv_root_c2 = (float)(1.0 / sqrt(c2));
  const int64_t span = d.state_bits == 32 ? SPAN32 : SPAN8;
  int k = 0;
  int64_t done = 0;  // pieces of tensor k
  while (k < n) {
    int64_t groups = 0;
    a.n = 0;
    a.place = k;
    a.done = done;
    // a run of tensors, the last of which the next launch may go on with; an
    // empty one takes no workgroup (a place in the table keeps the numbering)
    while (k < n && a.n < TENSORS && groups < GROUPS) {
      const tp_adamw_tensor& x = t[k];
      const int64_t left = (x.count + span - 1) / span - done;
      const int64_t now = left < GROUPS - groups ? left : GROUPS - groups;
      a.first[a.n] = (int)groups;
      a.t[a.n++] = Tensor{x.param, (bf16_t*)x.param_bf16, x.grad, x.m, x.v, x.m_scale, x.v_scale,
                          x.count, x.weight_decay};
      groups += now;
      done += now;
      if (now < left) break;
      ++k;
      done = 0;
    }
    if (groups == 0) continue;
    const bool bf = d.grad_dtype == TP_BF16;
    if (d.state_bits == 32) {
      if (bf) hipLaunchKernelGGL(step32_kernel<bf16_t>, dim3((unsigned)groups), dim3(NT), 0, st, a);
      else hipLaunchKernelGGL(step32_kernel<float>, dim3((unsigned)groups), dim3(NT), 0, st, a);
    } else {
      if (bf) hipLaunchKernelGGL(step8_kernel<bf16_t>, dim3((unsigned)groups), dim3(NT), 0, st, a);
      else hipLaunchKernelGGL(step8_kernel<float>, dim3((unsigned)groups), dim3(NT), 0, st, a);
    }
    const hipError_t he = hipGetLastError();
    if (he != hipSuccess) return he;
  }
  return hipSuccess;
}

}  // namespace tpmlp
