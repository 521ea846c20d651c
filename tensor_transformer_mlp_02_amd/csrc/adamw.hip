// AdamW over many tensors (Megatron-LM 源码精读——大模型并行训练全景 §五: fp32
// main parameters and gradients, bf16 weights).  Per element
//   m = b1 m + (1-b1) g,  v = b2 v + (1-b2) g^2,
//   p = p (1 - lr wd) - lr/c1 * m / (sqrt(v)/sqrt(c2) + eps)
// Nothing is reused: the kernel is HBM-bound at 30 bytes an element with
// fp32 states (fp32 gradient, bf16 copy) and 18 with 8-bit ones.
//
// The tensors travel by value in the kernel's arguments, up to CHUNK_TENSORS
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
constexpr int TENSORS = 48;        // of one launch: the arguments stay under 4 KiB
constexpr int SPAN = 4096;         // elements of one workgroup's piece of a tensor
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
  int first;  // workgroup of its first piece
};

struct Args {
  Tensor t[TENSORS];
  int n, place;  // tensors here; place of the first in the caller's list
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

__device__ __forceinline__ int find_tensor(const Args& A, int b) {
  int lo = 0, hi = A.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (A.t[mid].first <= b) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float load_grad(const float* g, int64_t i) { return g[i]; }
__device__ __forceinline__ float load_grad(const bf16_t* g, int64_t i) { return bf16_to_f32(g[i]); }

__device__ __forceinline__ float new_param(float p, float m, float root, const Scalars& s) {
  return p * s.decay - s.step_size * (m / (root * s.inv_root_c2 + s.eps));
}

// fp32 states
template <typename GT>
__global__ __launch_bounds__(NT) void step32_kernel(Args A) {
  const int k = find_tensor(A, blockIdx.x);
  const Tensor& t = A.t[k];
  Scalars s;
  if (!scalars(A, k, s)) return;
  const int64_t i0 = (int64_t)(blockIdx.x - t.first) * SPAN;
  const int64_t i1 = min(i0 + SPAN, t.count);
  const GT* grad = reinterpret_cast<const GT*>(t.g);
  float* mp = reinterpret_cast<float*>(t.m);
  float* vp = reinterpret_cast<float*>(t.v);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += NT) {
    const float g = load_grad(grad, i) * s.gs;
    const float m = mp[i] * A.b1 + g * A.omb1;
    const float v = vp[i] * A.b2 + g * g * A.omb2;
    const float p = new_param(t.p[i], m, sqrtf(v), s);
    mp[i] = m;
    vp[i] = v;
    t.p[i] = p;
    if (t.p16) t.p16[i] = f32_to_bf16(p);
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x = max(x, (uint32_t)__shfl_xor((int)x, d, 64));
  return x;
}

// scale and its inverse of a block whose largest magnitude has these bits
// (bits of non-negative floats order like the floats, NaN above all).  An
// infinity makes the scale NaN, like a NaN: the block's state says so.
__device__ __forceinline__ void block_scale(uint32_t bits, float& scale, float& inv) {
  const float top = __uint_as_float(bits);
  const bool none = top <= 0x1p-100f;
  scale = none ? 0.f : bits >= 0x7f800000u ? __builtin_nanf("") : top / FMAX;
  inv = top > 0x1p-100f ? FMAX / top : 0.f;
}

// t rounded to an E4M3 value, down or up by chance u in [0, 1).  The step
// between neighbouring values at |t| in [2^k, 2^(k+1)) is 2^(k-3), and 2^-9
// below 2^-6.
//   a plain value: floor(t + u) in steps, t on average
//   a root: up from k steps with the chance (t^2 - k^2) / ((k+1)^2 - k^2),
//     so that its square, the second moment, is kept on average (a root kept
//     on average would add the rounding's variance to v at every step); a
//     positive one never becomes 0
// The variance that this adds stays small: a state that moves by d steps of
// its code is moved up or down with a chance of about d.
template <bool ROOT>
__device__ __forceinline__ float round_e4m3(float t, float u, bool positive) {
  const uint32_t e = max((__float_as_uint(t) >> 23) & 0xffu, 121u) - 3u;  // biased exponent of it
  t = t * __uint_as_float((254u - e) << 23);
  float k;
  if constexpr (ROOT) {
    k = floorf(t);
    const float odd = 2.f * k + 1.f;
    k += (t - k) * (t + k) + u * odd >= odd ? 1.f : 0.f;
    if (positive) k = fmaxf(k, 1.f);
  } else {
    k = floorf(t + u);
  }
  k = k * __uint_as_float(e << 23);
  return k > FMAX ? FMAX : k < -FMAX ? -FMAX : k;  // NaN stays NaN
}

// 8-bit states: a wavefront takes a block of 256, four neighbours a lane
template <typename GT>
__global__ __launch_bounds__(NT) void step8_kernel(Args A) {
  const int k = find_tensor(A, blockIdx.x);
  const Tensor& t = A.t[k];
  Scalars s;
  if (!scalars(A, k, s)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i0 = (int64_t)(blockIdx.x - t.first) * SPAN;
  const int64_t i1 = min(i0 + SPAN, t.count);
  const GT* grad = reinterpret_cast<const GT*>(t.g);
  uint8_t* mc = reinterpret_cast<uint8_t*>(t.m);
  uint8_t* vc = reinterpret_cast<uint8_t*>(t.v);
  for (int64_t b0 = i0 + wave * BLOCK; b0 < i1; b0 += (NT / 64) * BLOCK) {
    const int64_t blk = b0 / BLOCK;
    const float ms = t.ms[blk], vs = t.vs[blk];
    float m[4], r[4];
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = b0 + lane * 4 + j;
      m[j] = r[j] = 0.f;
      if (i < i1) {
        const float g = load_grad(grad, i) * s.gs;
        const float mo = __builtin_amdgcn_cvt_f32_fp8((int)mc[i], 0) * ms;
        const float ro = __builtin_amdgcn_cvt_f32_fp8((int)vc[i], 0) * vs;
        m[j] = mo * A.b1 + g * A.omb1;
        r[j] = sqrtf(ro * ro * A.b2 + g * g * A.omb2);
        const float p = new_param(t.p[i], m[j], r[j], s);
        t.p[i] = p;
        if (t.p16) t.p16[i] = f32_to_bf16(p);
      }
      mtop = max(mtop, __float_as_uint(m[j]) & 0x7fffffffu);
      vtop = max(vtop, __float_as_uint(r[j]) & 0x7fffffffu);
    }
    float msc, minv, vsc, vinv;
    block_scale(wave_max(mtop), msc, minv);
    block_scale(wave_max(vtop), vsc, vinv);
    if (lane == 0) {
      t.ms[blk] = msc;
      t.vs[blk] = vsc;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = b0 + lane * 4 + j;
      if (i < i1) {
        const uint32_t h = mix(((uint32_t)i ^ s.key) + (uint32_t)(i >> 32));
        const float um = (float)(h & 0xffffu) * 0x1p-16f, ur = (float)(h >> 16) * 0x1p-16f;
        const float cm = round_e4m3<false>(m[j] * minv, um, false);
        const float cr = round_e4m3<true>(r[j] * vinv, ur, r[j] > 0.f);
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(cm, cr, 0, false);
        mc[i] = (uint8_t)(w & 0xff);
        vc[i] = (uint8_t)((w >> 8) & 0xff);
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
  int k = 0;
  while (k < n) {
    int64_t groups = 0;
    a.n = 0;
    a.place = k;
    // a run of tensors; an empty one takes no workgroup (a place in the
    // table keeps the numbering)
    for (; k < n && a.n < TENSORS; ++k) {
      const tp_adamw_tensor& x = t[k];
      const int64_t pieces = (x.count + SPAN - 1) / SPAN;
      if (groups + pieces > 0x7fffffff) break;
      a.t[a.n++] = Tensor{x.param, (bf16_t*)x.param_bf16, x.grad, x.m, x.v, x.m_scale, x.v_scale,
                          x.count, x.weight_decay, (int)groups};
      groups += pieces;
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
