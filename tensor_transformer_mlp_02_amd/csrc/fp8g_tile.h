// Products of 8-bit codes with group scales on the matrix cores (the
// formulas: include/tpmlp_fp8g.h).  MFMA-bound.
//
// A workgroup makes a tile of (16 FM WM) x (16 FN WN) outputs with WM x WN
// wavefronts, each 16 FM x 16 FN as FM x FN blocks.  A k-tile is one group of 128.
//   SUM_FP8  v_mfma_f32_16x16x128_f8f6f4 makes a block's sum over the group in one
//            instruction: scaled and added in fp32 a step later (TP_GROUP_F32), or the
//            instruction applies the scales itself and accumulates (TP_GROUP_E8M0).
//   SUM_F32  codes are widened to bf16 (E8M0 scales go into the exponents) for four
//            v_mfma_f32_16x16x32_bf16, whose sums are fp32's.
// 4096 x 8192 x 3584: SUM_FP8 119 to 125 us (2.0 PFLOP/s; E8M0 scales 112 to 118), SUM_F32 206 (E8M0 194).
// The matrix cores are busy 42 % of the time; the rest is waiting at the barrier and for the
// columns of each k-tile, and the widening beside SUM_F32's instructions.
//
// Block i's row index a is row FM a + i of the wavefront's, block j's column
// index b is column 16 j + b.  The instruction is issued with the B codes first, which
// leaves a lane (p = lane % 16, q = lane / 16) with row index p and column indices
// 4 q .. 4 q + 3: in all FM neighbouring rows x 4 neighbouring columns of each block j.  So
// outputs are stored without a turn through shared memory, a lane's row scales are neighbours,
// and with FM = 8 a group of 128 tokens is one wavefront's (its largest magnitude a
// reduction over 16 lanes) and the codes of a transposed output are 8 bytes a lane.
//
// Shared memory holds rows of 128 codes, the 16-byte chunk c of a row at
// c ^ (the row's index a or b) % 8: the 8 lanes that are served together read 8
// different chunks.  A lane takes chunks q and q + 4 (the order of the summed index is free,
// as long as A and B agree; 2 q and 2 q + 1 meet half as many bank conflicts again, 2.5 % of
// the time of 4096 x 8192 x 3584; with none left it is no faster).  Row scales lie by step: that
// of row FM a + i at 16 i + a.
#pragma once

#include "fp8g.h"

namespace tpmlp {
namespace g8 {

// How a group's products are added: by the FP8 instruction, or widened to bf16
enum { SUM_FP8 = 0, SUM_F32 = 1 };
// G_RAW_*: the gated block's fp32 values, for a quantization of their own
enum { G_STORE = 0, G_GLU_FWD = 1, G_GLU_BWD = 2, G_RAW_FWD = 3, G_RAW_BWD = 4 };

template <int FMT_A, int FMT_B, int OB>  // OB: sb's byte; sa's is the first
__device__ __forceinline__ f32x4_t mfma_scaled(i32x8_t b, i32x8_t a, f32x4_t c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FMT_B, FMT_A, OB, sb, 0, sa);
}
template <int FMT_A, int FMT_B>
__device__ __forceinline__ f32x4_t mfma_plain(i32x8_t b, i32x8_t a, f32x4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FMT_B, FMT_A, 0, 0, 0, 0);
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void_t;

// a buffer of so many bytes: what is read behind its end is zeros
__device__ __forceinline__ rsrc_t buffer_of(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, 0x00020000);
}
struct Place {
  int64_t m0;  // first row of the wavefront
  int n0;      // first column of the workgroup's tile (of F, in the gated forward)
  int wm, wn, p, q;
};

// Outputs go through buffers that end with the last row; a column past the
// last takes an offset behind every end.  So no output needs a branch.  (Both halves of
// [G|U] have a buffer: a scalar offset is taken off the size before the comparison,
// and a wavefront without rows has none to take it from.)
constexpr uint32_t OUTSIDE = 0x80000000u;
__device__ __forceinline__ u32x2_t bf16x4(f32x4_t v) {
  return (u32x2_t){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// acc[i][j][t]: row m0 + FM p + i; column 16 j + 4 q + t of the wavefront's
template <int WM, int WN, int FM, int FN>
__device__ __forceinline__ void store_plain(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[FM][FN]) {
  const int n = at.n0 + at.wn * 16 * FN + at.q * 4, size = a.out_bf16 ? 2 : 4;
  const int rows = (int)max((int64_t)0, min((int64_t)(16 * FM), a.M - at.m0));
  const rsrc_t rc = buffer_of(reinterpret_cast<uint8_t*>(a.C) + at.m0 * a.N * size, rows * a.N * size);
  auto offset = [&](int i, int j) {
    return n + 16 * j < a.N ? (uint32_t)((FM * at.p + i) * a.N + n + 16 * j) * size : OUTSIDE;
  };
  static_for<0, FM / 2>([&](auto Ic) {  // two rows' loads at a time
    constexpr int i0 = 2 * decltype(Ic)::value;
    if (a.accumulate) {
      f32x4_t c[2][FN];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          c[i][j] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rc, offset(i0 + i, j), 0, 0));
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i0 + i][j][t] += c[i][j][t];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if (a.out_bf16) __builtin_amdgcn_raw_buffer_store_b64(bf16x4(acc[i0 + i][j]), rc, offset(i0 + i, j), 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[i0 + i][j]), rc, offset(i0 + i, j), 0, 0);
      }
  });
}

// The gated block's values in fp32 (a.raw): their groups span tiles
template <int WM, int WN, int FM, int FN>
__device__ __forceinline__ void store_raw_fwd(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[FM][FN]) {
  constexpr int J = FN / 2;
  const int64_t F = a.N, f = at.n0 + at.wn * 8 * FN + at.q * 4;
  const Gate gate(a.gate);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = at.m0 + FM * at.p + i;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t c = f + 16 * j;
      if (c >= F) continue;
      float g[4], u[4], h[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        g[t] = acc[i][j][t];
        u[t] = acc[i][J + j][t];
        h[t] = gate.act(g[t]) * u[t];
      }
      if (a.Z) {
        Store4<bf16_t>::store(a.Z, m * 2 * F + c, g);
        Store4<bf16_t>::store(a.Z, m * 2 * F + F + c, u);
      }
      if (a.H) Store4<bf16_t>::store(a.H, m * F + c, h);
      if (a.raw) Store4<float>::store(a.raw, m * F + c, h);
    }
  }
}
template <int WM, int WN, int FM, int FN>
__device__ __forceinline__ void store_raw_bwd(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[FM][FN]) {
  const int64_t F = a.N, f = at.n0 + at.wn * 16 * FN + at.q * 4;
  const Gate gate(a.gate);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = at.m0 + FM * at.p + i;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t c = f + 16 * j;
      if (c >= F) continue;
      float g[4], u[4], dg[4], du[4];
      Store4<bf16_t>::load(a.Z, m * 2 * F + c, g);
      Store4<bf16_t>::load(a.Z, m * 2 * F + F + c, u);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float act, slope;
        gate.both(g[t], act, slope);
        dg[t] = acc[i][j][t] * u[t] * slope;
        du[t] = acc[i][j][t] * act;
      }
      Store4<float>::store(a.raw, m * 2 * F + c, dg);
      Store4<float>::store(a.raw, m * 2 * F + F + c, du);
    }
  }
}

// The 8 codes that a lane has of one column (its 8 rows; `top` the largest
// magnitude among them), by the largest over the wavefront's 128 rows
template <int FMT, int SC>
__device__ __forceinline__ void store_column(uint8_t* q_t, void* s_t, const float v[8], uint32_t top, int64_t pm,
                                             int64_t m, int64_t col, int64_t cols, int64_t token_group, int p) {
  const GroupScale<FMT, SC> gs(top_of_16(top));
  const u32x2_t o = {codes4<FMT>(v[0], v[1], v[2], v[3], gs.inv), codes4<FMT>(v[4], v[5], v[6], v[7], gs.inv)};
  if (col < cols) {
    *reinterpret_cast<u32x2_t*>(q_t + col * pm + m) = o;
    if (p == 0) gs.store(s_t, token_group * cols + col);
  }
}

// Gated forward: blocks j < FN/2 hold the gate, the others the up projection, of the
// same columns 16 (j mod FN/2) + 4 q + t.  The tile has 128 of them: one group.
template <int WM, int WN, int FN, int SC>
__device__ __forceinline__ void store_glu_fwd(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[8][FN],
                                              uint32_t* red) {
  constexpr int J = FN / 2;
  static_assert(8 * FN * WN == 128, "one group of 128 columns");
  const int F = a.N, pf = (int)padded(F);
  const int64_t pm = padded(a.M), m = at.m0 + 8 * at.p;
  const int f = at.n0 + at.wn * 8 * FN + at.q * 4;
  const int rows = (int)max((int64_t)0, min((int64_t)128, a.M - at.m0));
  const rsrc_t rz = buffer_of(reinterpret_cast<bf16_t*>(a.Z) + at.m0 * 2 * F, a.Z ? rows * F * 4 : 0);
  const rsrc_t rz2 = buffer_of(reinterpret_cast<bf16_t*>(a.Z) + (at.m0 * 2 + 1) * F, a.Z && rows ? (rows * 2 - 1) * F * 2 : 0);
  const rsrc_t rh = buffer_of(reinterpret_cast<bf16_t*>(a.H) + at.m0 * F, a.H ? rows * F * 2 : 0);
  const rsrc_t rq = buffer_of(a.q + at.m0 * pf, a.q ? rows * pf : 0);
  const Gate gate(a.gate);
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top[i] = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = f + 16 * j;
      const f32x4_t g = acc[i][j], u = acc[i][J + j];
      if (a.Z) {
        const uint32_t off = c < F ? (uint32_t)((8 * at.p + i) * 2 * F + c) * 2u : OUTSIDE;
        __builtin_amdgcn_raw_buffer_store_b64(bf16x4(g), rz, off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b64(bf16x4(u), rz2, off, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        acc[i][j][t] = gate.act(g[t]) * u[t];
        top[i] = max(top[i], mag(acc[i][j][t]));
      }
      if (a.H)
        __builtin_amdgcn_raw_buffer_store_b64(bf16x4(acc[i][j]), rh, c < F ? (uint32_t)((8 * at.p + i) * F + c) * 2u : OUTSIDE, 0, 0);
    }
  }
  if (a.q) {
    // the group's largest magnitude of each row: 4 lanes, then the wavefronts
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = xor_max(xor_max(top[i], 16), 32);
    uint32_t* mine = red + (at.wm * WN + at.wn) * 128;
    if (at.q == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[8 * at.p + i] = top[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t w = 0;
#pragma unroll
      for (int c = 0; c < WN; ++c) w = max(w, red[(at.wm * WN + c) * 128 + 8 * at.p + i]);
      const GroupScale<0, SC> gs(w);
#pragma unroll
      for (int j = 0; j < J; ++j)
        __builtin_amdgcn_raw_buffer_store_b32(codes4<0>(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], gs.inv), rq,
                                              (uint32_t)((8 * at.p + i) * pf + f + 16 * j), 0, 0);
      if (at.wn == 0 && at.q == 0 && m + i < a.M) gs.store(a.s, (int64_t)(at.n0 / kGroup) * a.M + m + i);
    }
  }
  if (a.q_t && at.m0 < pm) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        float v[8];
        uint32_t col = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = acc[i][j][t];
          col = max(col, mag(v[i]));
        }
        store_column<0, SC>(a.q_t, a.s_t, v, col, pm, m, f + 16 * j + t, F, at.m0 / kGroup, at.p);
      }
  }
}

// Gated backward: acc is dH; a lane has 4 neighbouring columns of F of each of FN
// blocks, taken block by block: dG and dU are formed from the saved G and U, and a column's codes
// can be made at once.  A row's wait for the largest of its group: of 4
// blocks the first two's dU waits in shared memory meanwhile, so that dG, dU and the
// dH that is left fit the registers.  A tile has whole groups of 128 columns, WG wavefronts each.
// Rows and columns past the last read as zeros and are not stored.
template <int WM, int WN, int FN>
constexpr int glu_bwd_shared() {  // bytes
  return WM * WN * (2 * 128 * 4 + (FN == 4 ? 64 * 64 * 4 : 0));
}
template <int WM, int WN, int FN, int FMT, int SC>
__device__ __forceinline__ void store_glu_bwd(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[8][FN],
                                              uint8_t* shared) {
  constexpr int WG = 128 / (16 * FN);          // wavefronts of a group of columns
  constexpr int C = 4, NH = FN, PARKED = FN == 4 ? 2 : 0;
  static_assert(WN % WG == 0 && (FN == 1 || FN == 4));
  const int wave = at.wm * WN + at.wn, lane = at.q * 16 + at.p;
  uint32_t* red = reinterpret_cast<uint32_t*>(shared);  // [dG|dU] of each wavefront's 128 rows
  f32x4_t* wait = reinterpret_cast<f32x4_t*>(shared + WM * WN * 1024) + (wave * 16) * 64 + lane;
  const int F = a.N, pf = (int)padded(F), gf = pf / kGroup;
  const int64_t pm = padded(a.M);
  const int f = at.n0 + at.wn * 16 * FN + at.q * 4;
  const int64_t m = at.m0 + 8 * at.p;
  const int rows = (int)max((int64_t)0, min((int64_t)128, a.M - at.m0));
  const rsrc_t rz = buffer_of(reinterpret_cast<const bf16_t*>(a.Z) + at.m0 * 2 * F, rows * F * 4);
  const rsrc_t rz2 = buffer_of(reinterpret_cast<const bf16_t*>(a.Z) + (at.m0 * 2 + 1) * F, rows ? (rows * 2 - 1) * F * 2 : 0);
  const rsrc_t rq = buffer_of(a.q + at.m0 * 2 * pf, a.q ? rows * pf * 2 : 0);
  const rsrc_t rq2 = buffer_of(a.q + (at.m0 * 2 + 1) * pf, a.q && rows ? (rows * 2 - 1) * pf : 0);
  const Gate gate(a.gate);
  const int64_t token_group = at.m0 / kGroup;
  const bool turned = a.q_t && at.m0 < pm;
  float dg[NH][8][C], du[NH][8][C];
  uint32_t rg[8], ru[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rg[i] = ru[i] = 0;
  static_for<0, NH>([&](auto Hc) {
    constexpr int hf = decltype(Hc)::value;
    const int c = f + 16 * hf;
    uint32_t cg[C] = {0, 0, 0, 0}, cu[C] = {0, 0, 0, 0};
    static_for<0, 2>([&](auto Ic) {  // four rows' loads at a time
      constexpr int i0 = 4 * decltype(Ic)::value;
      u32x2_t zg[4], zu[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t off = c < F ? (uint32_t)((8 * at.p + i0 + i) * 2 * F + c) * 2u : OUTSIDE;
        zg[i] = __builtin_amdgcn_raw_buffer_load_b64(rz, off, 0, 0);
        zu[i] = __builtin_amdgcn_raw_buffer_load_b64(rz2, off, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const float g = __uint_as_float(k & 1 ? zg[i][k / 2] & 0xffff0000u : zg[i][k / 2] << 16);
          const float u = __uint_as_float(k & 1 ? zu[i][k / 2] & 0xffff0000u : zu[i][k / 2] << 16);
          const float d = acc[i0 + i][hf][k];
          float act, slope;
          gate.both(g, act, slope);
          dg[hf][i0 + i][k] = d * u * slope;
          du[hf][i0 + i][k] = d * act;
          // (both maxima here and not put off: the magnitudes kept would take as many registers again)
          const uint32_t x = mag(dg[hf][i0 + i][k]), y = mag(du[hf][i0 + i][k]);
          rg[i0 + i] = max(rg[i0 + i], x);
          ru[i0 + i] = max(ru[i0 + i], y);
          cg[k] = max(cg[k], x);
          cu[k] = max(cu[k], y);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) asm volatile("" : "+v"(cg[k]), "+v"(cu[k]), "+v"(rg[i0 + k]), "+v"(ru[i0 + k]));
      __builtin_amdgcn_sched_barrier(0);
    });
    if (turned) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float v[8], w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = dg[hf][i][k];
          w[i] = du[hf][i][k];
        }
        store_column<FMT, SC>(a.q_t, a.s_t, v, cg[k], pm, m, c + k, F, token_group, at.p);
        store_column<FMT, SC>(a.q_t + F * pm, reinterpret_cast<uint8_t*>(a.s_t) + F * (pm / kGroup) * (SC == TP_GROUP_F32 ? 4 : 1),
                              w, cu[k], pm, m, c + k, F, token_group, at.p);
      }
    }
    if constexpr (hf < PARKED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) wait[(8 * hf + i) * 64] = (f32x4_t){du[hf][i][0], du[hf][i][1], du[hf][i][2], du[hf][i][3]};
    }
    __builtin_amdgcn_sched_barrier(0);
  });
  if (!a.q) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rg[i] = xor_max(xor_max(rg[i], 16), 32);
    ru[i] = xor_max(xor_max(ru[i], 16), 32);
    if (at.q == 0) {
      red[wave * 256 + 8 * at.p + i] = rg[i];
      red[wave * 256 + 128 + 8 * at.p + i] = ru[i];
    }
  }
  __syncthreads();
  // a row's largest over the wavefronts of its group
  const uint32_t* peers = red + (at.wm * WN + at.wn / WG * WG) * 256 + 8 * at.p;
  static_for<0, 8>([&](auto Ic) {
    constexpr int i = decltype(Ic)::value;
    uint32_t tg = 0, tu = 0;
#pragma unroll
    for (int k = 0; k < WG; ++k) {
      tg = max(tg, peers[k * 256 + i]);
      tu = max(tu, peers[k * 256 + 128 + i]);
    }
    const GroupScale<FMT, SC> sg(tg), su(tu);
    if (at.q == 0 && at.wn % WG == 0 && f < F && m + i < a.M) {
      sg.store(a.s, (int64_t)(f / kGroup) * a.M + m + i);
      su.store(a.s, (int64_t)(gf + f / kGroup) * a.M + m + i);
    }
    static_for<0, NH>([&](auto Hc) {
      constexpr int hf = decltype(Hc)::value;
      const int c = f + 16 * hf;
      const uint32_t off = c < pf ? (uint32_t)((8 * at.p + i) * 2 * pf + c) : OUTSIDE;
      if constexpr (hf < PARKED) {
        const f32x4_t w = wait[(8 * hf + i) * 64];
#pragma unroll
        for (int k = 0; k < 4; ++k) du[hf][i][k] = w[k];
      }
      const float *x = dg[hf][i], *y = du[hf][i];
      __builtin_amdgcn_raw_buffer_store_b32(codes4<FMT>(x[0], x[1], x[2], x[3], sg.inv), rq, off, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b32(codes4<FMT>(y[0], y[1], y[2], y[3], su.inv), rq2, off, 0, 0);
    });
  });
}

// ---- operands: memory -> shared memory -> registers --------------------------
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// The 32 codes of a block's row that a lane has, and the row's scale: asked
// for, and later waited for.  In between nothing may touch the registers
// (they have not arrived): what comes between is arithmetic on others.
struct Row {
  i32x4_t lo, hi;
  float s;
  template <int OFF>
  __device__ __forceinline__ void ask(uint32_t a0, uint32_t a1) {
    asm volatile("ds_read_b128 %0, %2 offset:%4\n\tds_read_b128 %1, %3 offset:%4"
                 : "=&v"(lo), "=&v"(hi) : "v"(a0), "v"(a1), "n"(OFF) : "memory");
  }
  template <int OFF, int SOFF>
  __device__ __forceinline__ void ask(uint32_t a0, uint32_t a1, uint32_t as) {
    asm volatile("ds_read_b128 %0, %3 offset:%6\n\tds_read_b128 %1, %4 offset:%6\n\tds_read_b32 %2, %5 offset:%7"
                 : "=&v"(lo), "=&v"(hi), "=&v"(s) : "v"(a0), "v"(a1), "v"(as), "n"(OFF), "n"(SOFF) : "memory");
  }
  __device__ __forceinline__ void wait_scale() {
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(lo), "+v"(hi), "+v"(s)::"memory");
  }
  __device__ __forceinline__ void arrived() { asm volatile("" : "+v"(lo), "+v"(hi)); }  // after a wait
  __device__ __forceinline__ void arrived_scale() { asm volatile("" : "+v"(lo), "+v"(hi), "+v"(s)); }
  __device__ __forceinline__ i32x8_t codes() const { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};

// Scales that a wavefront shares, through the scalar cache: their loads do
// not wait behind the operands' on their way to shared memory
typedef __attribute__((address_space(4))) const float const_float_t;
typedef __attribute__((address_space(4))) const uint32_t const_u32_t;
__device__ __forceinline__ float scalar_f32(const void* p, int64_t i) {
  return ((const_float_t*)(uintptr_t)p)[i];
}
// (the aligned word that a byte lies in: of a tensor's first and last bytes it holds up to 3 of others')
__device__ __forceinline__ uint32_t scalar_byte(const void* p, int64_t i) {
  const uintptr_t at = (uintptr_t)p + (uintptr_t)i;
  return (((const_u32_t*)(at & ~(uintptr_t)3))[0] >> (8 * (at & 3))) & 255u;
}

// The operands' tiles pass through NS buffers in shared memory: while one is
// multiplied, the next ones' loads (straight into shared memory) are on their way.
template <int WM, int WN, int FM, int FN, int NS, int SC, bool SQ, int FMT_A, int FMT_B, int SUM, int EPI>
__global__ __launch_bounds__(64 * WM * WN, WM * WN == 8 && FM * FN == 32 || FM == 4 ? 2 : 1) void gemm(G8GemmArgs a) {
  constexpr int BM = 16 * FM * WM, BN = 16 * FN * WN, NW = WM * WN;
  constexpr bool PAIR = EPI == G_GLU_FWD || EPI == G_RAW_FWD;
  static_assert(NS == 2 || NS == 3);
  static_assert(FM == 8 || (FM == 4 && EPI != G_GLU_FWD && EPI != G_GLU_BWD));
  static_assert(BM % 64 == 0 && BM % (8 * WM * WN) == 0 && BN % (8 * WM * WN) == 0);
  constexpr int COLS = PAIR ? BN / 2 : BN;  // columns of the output a tile has
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KiB loads of a wavefront (8 rows each)
  // Scales of rows, and E8M0 ones of columns, go by way of shared memory, a word each: a load
  // into registers is waited for together with all loads into shared memory before it.
  constexpr bool BLDS = SC == TP_GROUP_E8M0 && !SQ;
  constexpr int LOADS = LA + LB + 1 + (BLDS ? 1 : 0);
  // [A .. | B .. | row scales .. | column scales ..], NS of each
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, S_BYTES = BM * 4, SB_BYTES = BLDS ? BN * 4 : 0;
  constexpr int TILES = NS * (A_BYTES + B_BYTES + S_BYTES + SB_BYTES), LAST = EPI == G_GLU_BWD ? glu_bwd_shared<WM, WN, FN>() : 0;
  constexpr int SHARED = TILES > LAST ? TILES : LAST;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[SHARED];
  constexpr int B_AT = NS * A_BYTES, S_AT = B_AT + NS * B_BYTES, SB_AT = S_AT + NS * S_BYTES;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // tile: XCDs take contiguous runs, rastered in groups of 4 tile rows
  const int tile = a.first + xcd_logical_block(blockIdx.x, gridDim.x);
  const int group = tile / (4 * a.tiles_n), first = 4 * group;
  const int gm = min(4, a.tiles_m - first), li = tile - group * 4 * a.tiles_n;
  const int tm = first + li % gm, tn = li / gm;

  Place at;
  at.wm = wave / WN;
  at.wn = wave % WN;
  at.p = lane & 15;
  at.q = lane >> 4;
  const int64_t mt = (int64_t)tm * BM;
  at.m0 = mt + at.wm * 16 * FM;
  at.n0 = tn * COLS;

  const int kt_part = a.K / kGroup, kt_all = kt_part * a.parts;

  // a wavefront's loads, 8 rows each: lane l fills chunk l % 8 of row l / 8.  Each has a
  // buffer of its own, which begins at its first row's group: so the offsets are a
  // lane's alone (formed at each load they cost 4 % of 4096 x 8192 x 3584), and rows past the last
  // lie behind its end and read as zeros.
  const int lda = (int)a.lda;
  const int rows = (int)min((int64_t)BM, a.M - mt), cols = min(COLS, a.N - at.n0);
  const uint8_t* const from_a = a.A + mt * a.lda;
  const int l8 = lane >> 3, ch = lane & 7;
  const uint32_t va = l8 * lda, vb = l8 * a.K + ((ch ^ l8) << 4);
  const int slot = (wave % (BM / 64)) * 64 + lane;
  const int sr = slot / (16 * FM) * (16 * FM) + slot % 16 * FM + slot % (16 * FM) / 16;
  auto load_tile = [&](int kt, int buf) {
    const int part = kt >= kt_part ? 1 : 0, kb = kt - part * kt_part;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r0 = (wave * LA + i) * 8;
      const rsrc_t ra = buffer_of(from_a + r0 * lda + kt * 128, max(0, (rows - r0) * lda - kt * 128));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(lds + buf * A_BYTES + r0 * 128), 16,
                                               va + ((ch ^ ((r0 / FM + l8 / FM) & 7)) << 4), 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      // (gated forward: of a wavefront's rows the first half is the gate's)
      const int r0 = (wave * LB + i) * 8;
      const bool second = PAIR ? (r0 / (8 * FN)) % 2 == 1 : part == 1;
      const int n = PAIR ? r0 / (16 * FN) * (8 * FN) + r0 % (8 * FN) : r0;
      const rsrc_t rb = buffer_of((second ? a.B2 : a.B) + (int64_t)(at.n0 + n) * a.K + kb * 128, max(0, (cols - n) * a.K - kb * 128));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(lds + B_AT + buf * B_BYTES + r0 * 128), 16, vb, 0, 0, 0);
    }
    constexpr int W = SC == TP_GROUP_F32 ? 4 : 1;  // (bytes arrive as words)
    const rsrc_t rs = buffer_of(reinterpret_cast<const uint8_t*>(a.sA) + ((int64_t)kt * a.M + mt) * W, rows * W);
    lds_void_t* const to = (lds_void_t*)(lds + S_AT + buf * S_BYTES + (wave % (BM / 64)) * 256);
    if constexpr (W == 4) __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 4, sr * 4, 0, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, to, 1, sr, 0, 0, 0);
    if constexpr (BLDS) {
      const int n = (wave % (BN / 64)) * 64;
      const rsrc_t rsb = buffer_of(reinterpret_cast<const uint8_t*>(part ? a.sB2 : a.sB) + (int64_t)kb * a.N + at.n0, cols);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsb, (lds_void_t*)(lds + SB_AT + buf * SB_BYTES + n * 4), 1, n + lane, 0, 0, 0);
    }
  };

  // what a lane reads: chunks q and q + 4 of its rows
  const uint32_t l0 = lds_address(lds);
  const uint32_t c0 = (at.q ^ (at.p & 7)) << 4;
  const uint32_t pa = l0 + (at.wm * 16 * FM + FM * at.p) * 128 + c0, pb = l0 + B_AT + (at.wn * 16 * FN + at.p) * 128 + c0;
  const uint32_t ps = l0 + S_AT + (at.wm * 16 * FM + at.p) * 4, psb = l0 + SB_AT + (at.wn * 16 * FN + at.p) * 4;

  // Scales of a tile's columns: shared ones by way of the scalar cache, fp32 ones of each
  // column (a lane's are neighbours) straight into registers; past the last column they read as zeros
  constexpr int SBT = SC == TP_GROUP_F32 && !SQ ? 4 : 1;
  struct Scales {
    float b[SC == TP_GROUP_F32 ? SBT : 1][SC == TP_GROUP_F32 ? FN : 1];
    uint32_t eb;  // byte j: block j's
  };
  const int nw = PAIR ? at.n0 + at.wn * 8 * FN : at.n0 + at.wn * 16 * FN;  // the wavefront's first column
  const int64_t square = (int64_t)(min(nw, a.N - 1) / kGroup) * kt_part;
  auto load_scales = [&](int kt, Scales& s) {
    const int part = kt >= kt_part ? 1 : 0, kb = kt - part * kt_part;
    auto from = [&](int j) { return PAIR ? (j < FN / 2 ? a.sB : a.sB2) : (part ? a.sB2 : a.sB); };
    if constexpr (SQ) {
      s.eb = 0;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (SC == TP_GROUP_F32) s.b[0][j] = scalar_f32(from(j), square + kb);
        else s.eb |= scalar_byte(from(j), square + kb) << (8 * j);
      }
    } else if constexpr (SC == TP_GROUP_F32) {
      const int cols_w = max(0, min(16 * FN, a.N - nw));
      const rsrc_t rs = buffer_of(reinterpret_cast<const float*>(from(0)) + (int64_t)kb * a.N + nw, cols_w * 4);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const u32x4_t w = __builtin_amdgcn_raw_buffer_load_b128(rs, (16 * j + 4 * at.q) * 4, 0, 0);
#pragma unroll
        for (int t = 0; t < 4; ++t) s.b[t][j] = __uint_as_float(w[t]);
      }
    }
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

  Scales sc, sc_next;
  load_scales(0, sc_next);
  static_for<0, NS>([&](auto T) {
    if (decltype(T)::value < kt_all) load_tile(decltype(T)::value, decltype(T)::value);
  });
  // waits until at most `tiles` of the newest tiles' loads are on their way
  auto wait_tiles = [&](int tiles) {
    if (NS > 2 && tiles == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * 2) : "memory");
    else if (tiles == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  wait_tiles(min(kt_all, NS) - 1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  Row ra0, ra1;  // the rows of two steps in turn
  i32x8_t fb[SUM == SUM_FP8 ? FN : 1];
  bf16x8g_t wb[SUM == SUM_F32 ? FN : 1][4];
  auto byte_of = [](const Row& r) { return __float_as_uint(r.s); };  // a scale's, which arrived as a word
  auto widen_b = [&](auto J, const Row& r, const Scales& s) {
    constexpr int j = decltype(J)::value;
    const i32x8_t f = r.codes();
    if constexpr (SUM == SUM_FP8) {
      fb[j] = f;
    } else {
      const float e = SC == TP_GROUP_F32 ? 1.0f : e8m0_half(BLDS ? byte_of(r) : (s.eb >> (8 * j)) & 255);
#pragma unroll
      for (int c = 0; c < 4; ++c) wb[j][c] = widen<FMT_B>(f[2 * c], f[2 * c + 1], e);
    }
  };
  auto ask_a = [&](auto I, Row& r, int buf) {
    constexpr int i = decltype(I)::value;
    const uint32_t a0 = pa + buf * A_BYTES;
    r.template ask<i * 128, i * 64>(a0, a0 ^ 64, ps + buf * S_BYTES);
  };
  auto ask_columns = [&](Row (&b)[FN], int buf) {
    const uint32_t b0 = pb + buf * B_BYTES;
    static_for<0, FN>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (BLDS) b[j].template ask<j * 2048, j * 64>(b0, b0 ^ 64, psb + buf * SB_BYTES);
      else b[j].template ask<j * 2048>(b0, b0 ^ 64);
    });
  };
  // (all reads have been waited for)
  auto take_columns = [&](Row (&b)[FN], Scales& s) {
    if constexpr (BLDS) s.eb = 0;
    static_for<0, FN>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (BLDS) {
        b[j].arrived_scale();
        s.eb |= byte_of(b[j]) << (8 * j);
      } else {
        b[j].arrived();
      }
    });
    static_for<0, FN>([&](auto J) { widen_b(J, b[J], s); });
  };
  Row cb[FN];  // the wavefront's columns of a tile, on their way

  f32x4_t p[FN];
  float sa = 0.0f;
  auto add_group = [&](auto I, auto J) {
    constexpr int i = decltype(I)::value, j = decltype(J)::value;
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(p[j][t], sa * sc.b[SQ ? 0 : t][j], acc[i][j][t]);
    asm volatile("" : "+v"(acc[i][j]));  // (put off past the barrier, it would hold its registers)
  };

  if constexpr (FM == 4) {
    // A small tile: there are registers for all that a wavefront reads of it
    // and of the next, asked for together a tile ahead (one at a time, their
    // latencies were most of a tile's time)
    struct Set {
      Row a[FM], b[FN];
    };
    Set even, odd;
    auto ask_set = [&](Set& t, int buf) {
      ask_columns(t.b, buf);
      static_for<0, FM>([&](auto I) { ask_a(I, t.a[I], buf); });
    };
    auto wait_set = [&](Set& t) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      static_for<0, FN>([&](auto J) {
        if constexpr (BLDS) t.b[J].arrived_scale();
        else t.b[J].arrived();
      });
      static_for<0, FM>([&](auto I) { t.a[I].arrived_scale(); });
    };
    auto one_tile = [&](Set& t, Set& next, int kt, int buf, int buf_next) {
      sc = sc_next;
      load_scales(min(kt + 1, kt_all - 1), sc_next);
      // this tile is read, and the next one there, for every wavefront
      wait_tiles(max(0, min(kt_all - 2 - kt, NS - 2)));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      ask_set(next, buf_next);  // (behind the last tile: what nothing uses)
      if (kt + NS < kt_all) load_tile(kt + NS, buf);
      take_columns(t.b, sc);
      static_for<0, FM>([&](auto I) {
        constexpr int i = decltype(I)::value;
        const i32x8_t fa = t.a[i].codes();
        if constexpr (SUM == SUM_F32) {
          float e = 1.0f;
          if constexpr (SC == TP_GROUP_E8M0) e = e8m0_half(byte_of(t.a[i]));
          f32x4_t g[FN];
          static_for<0, 4>([&](auto Cc) {
            constexpr int c = decltype(Cc)::value;
            const bf16x8g_t wa = widen<FMT_A>(fa[2 * c], fa[2 * c + 1], e);
            static_for<0, FN>([&](auto J) {
              constexpr int j = decltype(J)::value;
              if constexpr (SC == TP_GROUP_E8M0) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][c], wa, acc[i][j], 0, 0, 0);
              else g[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][c], wa, c ? g[j] : (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
            });
          });
          if constexpr (SC == TP_GROUP_F32) {
            static_for<0, FN>([&](auto J) {
              constexpr int j = decltype(J)::value;
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[i][j][k] = fmaf(g[j][k], t.a[i].s * sc.b[SQ ? 0 : k][j], acc[i][j][k]);
            });
          }
        } else {
          static_for<0, FN>([&](auto J) {
            constexpr int j = decltype(J)::value;
            if constexpr (SC == TP_GROUP_F32) {
              const f32x4_t g = mfma_plain<FMT_A, FMT_B>(fb[j], fa, (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[i][j][k] = fmaf(g[k], t.a[i].s * sc.b[SQ ? 0 : k][j], acc[i][j][k]);
            } else {
              acc[i][j] = mfma_scaled<FMT_A, FMT_B, j>(fb[j], fa, acc[i][j], (int)sc.eb, (int)byte_of(t.a[i]));
            }
          });
        }
      });
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
      __builtin_amdgcn_sched_barrier(0);
      wait_set(next);  // (here: on their way round the loop they might be moved)
    };
    auto after = [](int buf) { return buf + 1 == NS ? 0 : buf + 1; };
    ask_set(even, 0);
    wait_set(even);
    int buf = 0, kt = 0;
    for (; kt + 1 < kt_all; kt += 2) {
      one_tile(even, odd, kt, buf, after(buf));
      buf = after(buf);
      one_tile(odd, even, kt + 1, buf, after(buf));
      buf = after(buf);
    }
    if (kt < kt_all) one_tile(even, odd, kt, buf, after(buf));
  } else {
    int buf = 0;
    sc = sc_next;
    ask_columns(cb, 0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    take_columns(cb, sc);
    ask_a(std::integral_constant<int, 0>{}, ra0, 0);
    for (int kt = 0; kt < kt_all; ++kt) {
      const bool more = kt + 1 < kt_all;
      const int buf_next = buf + 1 == NS ? 0 : buf + 1;
      load_scales(more ? kt + 1 : kt, sc_next);
      static_for<0, FM>([&](auto I) {
        constexpr int i = decltype(I)::value;
        Row& r = i & 1 ? ra1 : ra0;
        Row& next = i & 1 ? ra0 : ra1;
        r.wait_scale();
        if constexpr (i < FM - 1) {
          ask_a(std::integral_constant<int, (i + 1) % FM>{}, next, buf);
        } else {
          // the tile is read; the next one is there for every wavefront after
          // this, and the buffer takes the one NS on
          wait_tiles(max(0, min(kt_all - 2 - kt, NS - 2)));
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
          // (behind the last tile: rows that nothing uses, so that every path asks)
          ask_a(std::integral_constant<int, 0>{}, next, buf_next);
        }
        const i32x8_t fa = r.codes();
        // fp32 scales: a step's group sums are scaled and added during the next
        // step, when the instructions that make them have ended
        if constexpr (SUM == SUM_F32) {
          float e = 1.0f;
          if constexpr (SC == TP_GROUP_E8M0) e = e8m0_half(byte_of(r));
          static_for<0, 4>([&](auto Cc) {
            constexpr int c = decltype(Cc)::value;
            const bf16x8g_t wa = widen<FMT_A>(fa[2 * c], fa[2 * c + 1], e);
            static_for<0, FN>([&](auto J) {
              constexpr int j = decltype(J)::value;
              if constexpr (SC == TP_GROUP_E8M0) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][c], wa, acc[i][j], 0, 0, 0);
              } else {
                if constexpr (c == 0 && i > 0) add_group(std::integral_constant<int, i - 1>{}, J);
                p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][c], wa, c ? p[j] : (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
              }
            });
            if constexpr (c % 2) __builtin_amdgcn_sched_barrier(0);  // (two widenings at a time hold fewer registers)
          });
        } else {
          static_for<0, FN>([&](auto J) {
            constexpr int j = decltype(J)::value;
            if constexpr (SC == TP_GROUP_F32) {
              if constexpr (i > 0) add_group(std::integral_constant<int, i - 1>{}, J);
              p[j] = mfma_plain<FMT_A, FMT_B>(fb[j], fa, (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f});
            } else {
              acc[i][j] = mfma_scaled<FMT_A, FMT_B, j>(fb[j], fa, acc[i][j], (int)sc.eb, (int)byte_of(r));
            }
          });
        }
        // (the matrix cores are at work meanwhile: before the step's products these loads cost the
        // gated forward and the weight gradient 3 %)
        if constexpr (i == FM - 1) {
          __builtin_amdgcn_sched_barrier(0);
          if (kt + NS < kt_all) load_tile(kt + NS, buf);
        }
        if constexpr (SC == TP_GROUP_F32) sa = r.s;
        if constexpr (SC == TP_GROUP_E8M0) {
#pragma unroll
          for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      // (widened, the columns leave no room for the next ones before here; FP8 ones
      // would, but asked for beside the step's rows they took 3 % longer)
      ask_columns(cb, buf_next);
      if constexpr (SC == TP_GROUP_F32) {
        static_for<0, FN>([&](auto J) { add_group(std::integral_constant<int, FM - 1>{}, J); });
      }
      sc = sc_next;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      take_columns(cb, sc);
      buf = buf_next;
    }
    ra0.wait_scale();
  }
  __syncthreads();

  if constexpr (SUM == SUM_F32 && SC == TP_GROUP_E8M0) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] *= E8M0_SUMS;
  }
  uint32_t* red = reinterpret_cast<uint32_t*>(lds);
  if constexpr (EPI == G_GLU_FWD) store_glu_fwd<WM, WN, FN, SC>(a, at, acc, red);
  else if constexpr (EPI == G_GLU_BWD) store_glu_bwd<WM, WN, FN, FMT_A, SC>(a, at, acc, lds);
  else if constexpr (EPI == G_RAW_FWD) store_raw_fwd<WM, WN, FM, FN>(a, at, acc);
  else if constexpr (EPI == G_RAW_BWD) store_raw_bwd<WM, WN, FM, FN>(a, at, acc);
  else store_plain<WM, WN, FM, FN>(a, at, acc);
}

template <int WM, int WN, int FM, int FN, int NS, int SC, bool SQ, int FMT_A, int FMT_B, int SUM, int EPI>
static hipError_t launch(G8GemmArgs& a, hipStream_t st) {
  constexpr int BM = 16 * FM * WM, BN = EPI == G_GLU_FWD || EPI == G_RAW_FWD ? 8 * FN * WN : 16 * FN * WN;
  const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  if (tm * tn > 0x7fffffff) return hipErrorInvalidValue;
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tn;
  return g8_in_launches(tm * tn, [&](int64_t first, int64_t count) {
    a.first = (int)first;
    hipLaunchKernelGGL((gemm<WM, WN, FM, FN, NS, SC, SQ, FMT_A, FMT_B, SUM, EPI>), dim3((unsigned)count), dim3(64 * WM * WN), 0,
                       st, a);
    return hipGetLastError();
  });
}

}  // namespace g8
}  // namespace tpmlp
