// Products of 8-bit codes with group scales on the matrix cores (the
// formulas: include/tpmlp_fp8g.h).  MFMA-bound.
//
// A workgroup makes a tile of (128 WM) x (16 FN WN) outputs with WM x WN
// wavefronts, each 128 x 16 FN as 8 x FN blocks of
// v_mfma_f32_16x16x128_f8f6f4: one instruction spans exactly one group of the
// summed index, so its result is the group's exact sum, scaled and added in
// fp32 (TP_GROUP_F32), or the instruction applies the scales itself and
// accumulates (TP_GROUP_E8M0).
//
// Rows and columns are dealt to the blocks so that a lane's outputs lie
// together: block i's row index a is row 8 a + i of the wavefront's 128,
// block j's column index b is column FN b + j.  The instruction is issued with
// the B codes first, which leaves a lane (p = lane % 16, q = lane / 16) with
// row index p and column indices 4 q .. 4 q + 3: in all 8 neighbouring rows x 4 FN
// neighbouring columns.  So outputs are stored without a turn through shared
// memory, a lane's 8 row scales are neighbours, a group of 128 tokens is one
// wavefront's (its largest magnitude a reduction over 16 lanes) and the codes
// of a transposed output are 8 bytes a lane.
//
// Shared memory holds rows of 128 codes, the 16-byte chunk c of a row at
// c ^ (the row's index a or b) % 8: the 8 lanes that are served together read 8
// different chunks.
#pragma once

#include "fp8g.h"

namespace tpmlp {
namespace g8 {

// How a group's products are added: by the FP8 instruction, or widened to bf16
enum { SUM_FP8 = 0, SUM_F32 = 1 };
enum { G_STORE = 0, G_GLU_FWD = 1, G_GLU_BWD = 2 };

template <int FMT_A, int FMT_B, int OA, int OB>
__device__ __forceinline__ f32x4_t mfma_scaled(i32x8_t b, i32x8_t a, f32x4_t c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FMT_B, FMT_A, OB, sb, OA, sa);
}
template <int FMT_A, int FMT_B>
__device__ __forceinline__ f32x4_t mfma_plain(i32x8_t b, i32x8_t a, f32x4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, FMT_B, FMT_A, 0, 0, 0, 0);
}

struct Place {
  int64_t m0;  // first row of the wavefront
  int n0;      // first column of the workgroup's tile (of F, in the gated forward)
  int wm, wn, p, q;
};

// acc[i][j][t]: row m0 + 8 p + i; column (4 q + t) FN + j of the wavefront's
template <int WM, int WN, int FN>
__device__ __forceinline__ void store_plain(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[8][FN]) {
  const int n = at.n0 + at.wn * 16 * FN + at.q * 4 * FN;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t m = at.m0 + 8 * at.p + i;
    if (m >= a.M) continue;
#pragma unroll
    for (int h = 0; h < FN; ++h) {  // 4 columns at a time (bf16: 8 where a lane has them)
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = acc[i][(4 * h + k) % FN][(4 * h + k) / FN];
      const int64_t off = m * a.N + n + 4 * h;
      if (n + 4 * h >= a.N) continue;
      if (a.out_bf16) {
        Store4<bf16_t>::store(a.C, off, v);
      } else {
        if (a.accumulate) {
          float w[4];
          Store4<float>::load(a.C, off, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] += w[k];
        }
        Store4<float>::store(a.C, off, v);
      }
    }
  }
}

// The 8 codes that a lane has of one column (its 8 rows), from the column's
// largest magnitude over the wavefront's 128 rows
template <int FMT, int SC>
__device__ __forceinline__ void store_column(uint8_t* q_t, void* s_t, const float v[8], int64_t pm, int64_t m,
                                             int64_t col, int64_t cols, int64_t token_group, int p) {
  uint32_t top = mag(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = max(top, mag(v[i]));
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = xor_max(top, d);
  const GroupScale<FMT, SC> gs(top);
  const u32x2_t o = {codes4<FMT>(v[0], v[1], v[2], v[3], gs.inv), codes4<FMT>(v[4], v[5], v[6], v[7], gs.inv)};
  if (col < cols) {
    *reinterpret_cast<u32x2_t*>(q_t + col * pm + m) = o;
    if (p == 0) gs.store(s_t, token_group * cols + col);
  }
}

// Gated forward: blocks j < FN/2 hold the gate, the others the up projection, of the
// same columns f = (4 q + t) FN/2 + j: 2 FN neighbouring ones.  The tile has 128 of them: one
// group.
template <int WM, int WN, int FN, int SC>
__device__ __forceinline__ void store_glu_fwd(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[8][FN],
                                              uint32_t* red) {
  constexpr int J = FN / 2, C = 2 * FN;
  static_assert(8 * FN * WN == 128 && (C == 8 || C == 4), "one group of 128 columns");
  const int64_t F = a.N, pf = padded(F), pm = padded(a.M);
  const int fl = at.wn * 8 * FN + at.q * C;
  const int64_t f = at.n0 + fl;
  const int64_t m = at.m0 + 8 * at.p;
  const Gate gate(a.gate);
  auto put = [&](void* to, int64_t off, const float* v) {
    if constexpr (C == 8) Vec8<bf16_t>::store(to, off, v);
    else Store4<bf16_t>::store(to, off, v);
  };
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float h[C];
    if (a.Z && m + i < a.M && f < F) {
      float g[C], u[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        g[k] = acc[i][k % J][k / J];
        u[k] = acc[i][J + k % J][k / J];
      }
      put(a.Z, (m + i) * 2 * F + f, g);
      put(a.Z, (m + i) * 2 * F + F + f, u);
    }
    top[i] = 0;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      h[k] = gate.act(acc[i][k % J][k / J]) * acc[i][J + k % J][k / J];
      acc[i][k % J][k / J] = h[k];
      top[i] = max(top[i], mag(h[k]));
    }
    if (a.H && m + i < a.M && f < F) put(a.H, (m + i) * F + f, h);
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
      if (m + i < a.M) {
#pragma unroll
        for (int k = 0; k < C; k += 4)
          *reinterpret_cast<uint32_t*>(a.q + (m + i) * pf + f + k) =
              codes4<0>(acc[i][k % J][k / J], acc[i][(k + 1) % J][(k + 1) / J], acc[i][(k + 2) % J][(k + 2) / J],
                        acc[i][(k + 3) % J][(k + 3) / J], gs.inv);
        if (fl == 0) gs.store(a.s, (int64_t)(at.n0 / kGroup) * a.M + m + i);
      }
    }
  }
  if (a.q_t && at.m0 < pm) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = acc[i][k % J][k / J];
      store_column<0, SC>(a.q_t, a.s_t, v, pm, m, f + k, F, at.m0 / kGroup, at.p);
    }
  }
}

// Gated backward: acc is dH; a lane has 4 FN neighbouring columns of F, taken 8
// (or all) at a time.  dG and dU are formed twice from the saved G and U: for
// the groups' largest magnitudes, then for the codes (kept, they would take
// twice the registers of dH).  The multipliers of rows and columns wait in
// shared memory.  A tile has whole groups of 128 columns, WG wavefronts each.
template <int WM, int WN, int FN, int FMT, int SC>
__device__ __forceinline__ void store_glu_bwd(const G8GemmArgs& a, const Place& at, f32x4_t (&acc)[8][FN],
                                              uint32_t* red) {
  constexpr int WG = 128 / (16 * FN);          // wavefronts of a group of columns
  constexpr int C = 4 * FN < 8 ? 4 * FN : 8;   // columns at a time
  constexpr int NH = 4 * FN / C;
  static_assert(WN % WG == 0 && NH >= 1);
  // [dG|dU] of a row of a wavefront's 128; then [dG|dU] multipliers of its 16 FN columns
  constexpr int ROWS = 2 * 128, COLSX = 2 * 16 * FN;
  uint32_t* rows = red + (at.wm * WN + at.wn) * (ROWS + COLSX);
  float* cols = reinterpret_cast<float*>(rows + ROWS);
  const int64_t F = a.N, pf = padded(F), pm = padded(a.M), gf = pf / kGroup;
  const int64_t f = at.n0 + at.wn * 16 * FN + at.q * 4 * FN;
  const int64_t m = at.m0 + 8 * at.p;
  const Gate gate(a.gate);
  auto form = [&](int i, int hf, float* dg, float* du) {
    // (past the last row or column: another's G and U, and zeros)
    const int64_t c = f + C * hf, row = min(m + i, a.M - 1) * 2 * F + min(c, F - C);
    const bool there = m + i < a.M && c < F;
    float g[C], u[C];
    if constexpr (C == 8) {
      Vec8<bf16_t>::load(a.Z, row, g);
      Vec8<bf16_t>::load(a.Z, row + F, u);
    } else {
      Store4<bf16_t>::load(a.Z, row, g);
      Store4<bf16_t>::load(a.Z, row + F, u);
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const float d = acc[i][(C * hf + k) % FN][(C * hf + k) / FN];
      float act, slope;
      gate.both(g[k], act, slope);
      dg[k] = there ? d * u[k] * slope : 0.0f;
      du[k] = there ? d * act : 0.0f;
    }
  };
  const int64_t token_group = at.m0 / kGroup;
  const bool turned = a.q_t && at.m0 < pm;
  uint32_t rg[8], ru[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rg[i] = ru[i] = 0;
#pragma unroll
  for (int hf = 0; hf < NH; ++hf) {
    uint32_t cg[C], cu[C];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float dg[C], du[C];
      form(i, hf, dg, du);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const uint32_t x = mag(dg[k]), y = mag(du[k]);
        rg[i] = max(rg[i], x);
        ru[i] = max(ru[i], y);
        cg[k] = i ? max(cg[k], x) : x;
        cu[k] = i ? max(cu[k], y) : y;
      }
      if (i & 1) {  // (a few rows' loads at a time)
        asm volatile("" : "+v"(rg[i]), "+v"(ru[i])::"memory");
#pragma unroll
        for (int k = 0; k < C; ++k) asm volatile("" : "+v"(cg[k]), "+v"(cu[k]));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (a.q_t) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
          cg[k] = xor_max(cg[k], d);
          cu[k] = xor_max(cu[k], d);
        }
        if (at.p == 0) {
          const GroupScale<FMT, SC> sg(cg[k]), su(cu[k]);
          cols[at.q * 4 * FN + C * hf + k] = sg.inv;
          cols[16 * FN + at.q * 4 * FN + C * hf + k] = su.inv;
          const int64_t c = f + C * hf + k;
          if (turned && c < F) {
            sg.store(a.s_t, token_group * F + c);
            su.store(a.s_t, (pm / kGroup + token_group) * F + c);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rg[i] = xor_max(xor_max(rg[i], 16), 32);
    ru[i] = xor_max(xor_max(ru[i], 16), 32);
    if (at.q == 0) {
      rows[8 * at.p + i] = rg[i];
      rows[128 + 8 * at.p + i] = ru[i];
    }
  }
  __syncthreads();
  // a row's largest over the wavefronts of its group
  const uint32_t* peers = red + (at.wm * WN + at.wn / WG * WG) * (ROWS + COLSX);
  auto row_scale = [&](int which, int i) {
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < WG; ++k) w = max(w, peers[k * (ROWS + COLSX) + which * 128 + 8 * at.p + i]);
    return GroupScale<FMT, SC>(w);
  };
  if (a.q && at.q == 0 && at.wn % WG == 0 && f < F) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (m + i < a.M) {
        const int64_t g = f / kGroup;
        row_scale(0, i).store(a.s, g * a.M + m + i);
        row_scale(1, i).store(a.s, (gf + g) * a.M + m + i);
      }
  }
#pragma unroll
  for (int hf = 0; hf < NH; ++hf) {
    const int64_t c = f + C * hf;
    uint32_t og[C][2], ou[C][2];  // codes of C columns: 8 rows in two words
#pragma unroll
    for (int i2 = 0; i2 < 4; ++i2) {
      float dg[2][C], du[2][C];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 2 * i2 + i;
        form(r, hf, dg[i], du[i]);
        if (a.q && m + r < a.M && c < pf) {
          const float ig = row_scale(0, r).inv, iu = row_scale(1, r).inv;
          uint8_t* o = a.q + (m + r) * 2 * pf + c;
#pragma unroll
          for (int k = 0; k < C; k += 4) {
            *reinterpret_cast<uint32_t*>(o + k) = codes4<FMT>(dg[i][k], dg[i][k + 1], dg[i][k + 2], dg[i][k + 3], ig);
            *reinterpret_cast<uint32_t*>(o + pf + k) = codes4<FMT>(du[i][k], du[i][k + 1], du[i][k + 2], du[i][k + 3], iu);
          }
        }
      }
      if (a.q_t) {
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const float ig = cols[at.q * 4 * FN + C * hf + k], iu = cols[16 * FN + at.q * 4 * FN + C * hf + k];
          og[k][i2 / 2] = codes2<FMT>(dg[0][k], dg[1][k], ig, og[k][i2 / 2], i2 & 1);
          ou[k][i2 / 2] = codes2<FMT>(du[0][k], du[1][k], iu, ou[k][i2 / 2], i2 & 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
    }
    if (turned) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if (c + k < F) {
          *reinterpret_cast<u32x2_t*>(a.q_t + (c + k) * pm + m) = (u32x2_t){og[k][0], og[k][1]};
          *reinterpret_cast<u32x2_t*>(a.q_t + (F + c + k) * pm + m) = (u32x2_t){ou[k][0], ou[k][1]};
        }
      }
    }
  }
}

// ---- operands: memory -> shared memory -> registers --------------------------
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void lds_void_t;

// a buffer of so many bytes: what is read behind its end is zeros
__device__ __forceinline__ rsrc_t buffer_of(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, 0x00020000);
}
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
  __device__ __forceinline__ void wait() { asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(lo), "+v"(hi)::"memory"); }
  __device__ __forceinline__ void wait_scale() {
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(lo), "+v"(hi), "+v"(s)::"memory");
  }
  __device__ __forceinline__ i32x8_t codes() const { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};

// Scales that a wavefront shares, through the scalar cache: their loads do
// not wait behind the operands' on their way to shared memory
typedef __attribute__((address_space(4))) const float const_float_t;
typedef __attribute__((address_space(4))) const uint32_t const_u32_t;
__device__ __forceinline__ float scalar_f32(const void* p, int64_t i) {
  return ((const_float_t*)(uintptr_t)p)[i];
}
__device__ __forceinline__ uint32_t scalar_byte(const void* p, int64_t i) {
  const uintptr_t at = (uintptr_t)p + (uintptr_t)i;
  return (((const_u32_t*)(at & ~(uintptr_t)3))[0] >> (8 * (at & 3))) & 255u;
}

// The operands' tiles pass through NS buffers in shared memory: while one is
// multiplied, the next ones' loads (straight into shared memory) are on their way.
template <int WM, int WN, int FN, int NS, int SC, bool SQ, int FMT_A, int FMT_B, int SUM, int EPI>
__global__ __launch_bounds__(64 * WM * WN, WM * WN == 8 && FN == 4 ? 2 : 1) void gemm(G8GemmArgs a) {
  constexpr int BM = 128 * WM, BN = 16 * FN * WN, NW = WM * WN;
  constexpr bool PAIR = EPI == G_GLU_FWD;
  constexpr int COLS = PAIR ? BN / 2 : BN;  // columns of the output a tile has
  constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KiB loads of a wavefront (8 rows each)
  constexpr bool SLDS = SC == TP_GROUP_F32;          // row scales by way of shared memory
  constexpr int LOADS = LA + LB + (SLDS ? 1 : 0);
  // [A .. | B .. | row scales ..], NS of each
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, S_BYTES = SLDS ? BM * 4 : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * (A_BYTES + B_BYTES + S_BYTES)];
  constexpr int B_AT = NS * A_BYTES, S_AT = B_AT + NS * B_BYTES;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // tile: XCDs take contiguous runs, rastered in groups of 4 tile rows
  const int tile = xcd_logical_block(blockIdx.x, gridDim.x);
  const int group = tile / (4 * a.tiles_n), first = 4 * group;
  const int gm = min(4, a.tiles_m - first), li = tile - group * 4 * a.tiles_n;
  const int tm = first + li % gm, tn = li / gm;

  Place at;
  at.wm = wave / WN;
  at.wn = wave % WN;
  at.p = lane & 15;
  at.q = lane >> 4;
  const int64_t mt = (int64_t)tm * BM;
  at.m0 = mt + at.wm * 128;
  at.n0 = tn * COLS;

  const int kt_part = a.K / kGroup, kt_all = kt_part * a.parts;

  // a wavefront's loads: lane l fills chunk l % 8 of row 8 block + l / 8.
  // Rows past the last lie behind the buffer's end and read as zeros.  The
  // offsets are formed at each load, from two registers an operand.
  const int lda = (int)a.lda;
  const int rows = (int)min((int64_t)BM, a.M - mt), cols = min(COLS, a.N - at.n0);
  const rsrc_t ra = buffer_of(a.A + mt * a.lda, rows * lda);
  const rsrc_t rb = buffer_of(a.B + (int64_t)at.n0 * a.K, cols * a.K);
  const rsrc_t rb2 = buffer_of(a.B2 + (int64_t)at.n0 * a.K, cols * a.K);
  // shared rows of B: of a wavefront's 16 FN, block j's row b is row FN b + j;
  // gated forward: the gate's half of them, then the up projection's
  constexpr int RB = PAIR ? FN / 2 : FN;
  const int sr = (wave % (BM / 64)) * 64 + lane;
  auto load_tile = [&](int kt, int buf) {
    const int part = kt >= kt_part ? 1 : 0, kb = kt - part * kt_part;
    int ln = lane;
    asm volatile("" : "+v"(ln));  // (kept over the loop, each offset would be a register)
    const int l8 = ln >> 3, ch = ln & 7;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int blk = wave * LA + i;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(lds + buf * A_BYTES + blk * 1024), 16,
                                               (blk * 8 + l8) * lda + ((ch ^ (blk & 7)) << 4), kt * 128, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int r0 = (wave * LB + i) * 8, r = r0 + l8;
      const bool second = PAIR ? (r0 / (8 * FN)) % 2 == 1 : part == 1;
      const int n = PAIR ? r0 / (16 * FN) * (8 * FN) + r0 % (8 * FN) + l8 : r;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(second ? rb2 : rb, (lds_void_t*)(lds + B_AT + buf * B_BYTES + r0 * 128), 16,
                                               n * a.K + ((ch ^ ((r / RB) & 7)) << 4), kb * 128, 0, 0);
    }
    if constexpr (SLDS) {
      const rsrc_t rs = buffer_of(reinterpret_cast<const float*>(a.sA) + (int64_t)kt * a.M + mt, rows * 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (lds_void_t*)(lds + S_AT + buf * S_BYTES + (wave % (BM / 64)) * 256), 4, sr * 4, 0, 0, 0);
    }
  };

  // what a lane reads: chunks 2 q and 2 q + 1 of its rows
  const uint32_t l0 = lds_address(lds);
  const uint32_t c0 = ((2 * at.q) ^ (at.p & 7)) << 4;
  const uint32_t pa = l0 + (at.wm * 128 + 8 * at.p) * 128 + c0, pb = l0 + B_AT + (at.wn * 16 * FN + at.p * RB) * 128 + c0;
  const uint32_t ps = l0 + S_AT + (at.wm * 128 + 8 * at.p) * 4;

  // Scales of a tile: of its columns, and E8M0 ones of its rows.  Those of a
  // lane are neighbours, behind one offset from a base that a wavefront
  // shares; past the last row or column they read as zeros.
  constexpr int SBT = SC == TP_GROUP_F32 && !SQ ? 4 : 1;
  struct Scales {
    float b[SC == TP_GROUP_F32 ? SBT : 1][SC == TP_GROUP_F32 ? FN : 1];
    uint32_t eb, ea[2];
  };
  const int nw = PAIR ? at.n0 + at.wn * 8 * FN : at.n0 + at.wn * 16 * FN;  // the wavefront's first column
  const int rows_w = (int)max((int64_t)0, min((int64_t)128, a.M - at.m0)), cols_w = max(0, min(16 * FN, a.N - nw));
  const int64_t square = (int64_t)(min(nw, a.N - 1) / kGroup) * kt_part;
  auto load_scales = [&](int kt, Scales& s) {
    const int part = kt >= kt_part ? 1 : 0, kb = kt - part * kt_part;
    auto from = [&](int j) { return PAIR ? (j < FN / 2 ? a.sB : a.sB2) : (part ? a.sB2 : a.sB); };
    if constexpr (SC == TP_GROUP_F32) {
      if constexpr (SQ) {
#pragma unroll
        for (int j = 0; j < FN; ++j) s.b[0][j] = scalar_f32(from(j), square + kb);
      } else {
        const rsrc_t rs = buffer_of(reinterpret_cast<const float*>(from(0)) + (int64_t)kb * a.N + nw, cols_w * 4);
#pragma unroll
        for (int k = 0; k < 4 * FN; k += 4) {  // column FN t + j of the lane's 4 FN
          const u32x4_t w = __builtin_amdgcn_raw_buffer_load_b128(rs, (at.q * 4 * FN + k) * 4, 0, 0);
#pragma unroll
          for (int c = 0; c < 4; ++c) s.b[(k + c) / FN][(k + c) % FN] = __uint_as_float(w[c]);
        }
      }
    } else {
      s.eb = 0;
      if constexpr (SQ) {
#pragma unroll
        for (int j = 0; j < FN; ++j) s.eb |= scalar_byte(from(j), square + kb) << (8 * j);
      } else {
        const rsrc_t rs = buffer_of(reinterpret_cast<const uint8_t*>(from(0)) + (int64_t)kb * a.N + nw, cols_w);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          s.eb |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, at.p * FN + j, 0, 0) << (8 * j);
      }
      const rsrc_t rs = buffer_of(reinterpret_cast<const uint8_t*>(a.sA) + (int64_t)kt * a.M + at.m0, rows_w);
      s.ea[0] = s.ea[1] = 0;
      if (rows_w == 128) {
        const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(rs, 8 * at.p, 0, 0);
        s.ea[0] = w[0];
        s.ea[1] = w[1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          s.ea[i >> 2] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, 8 * at.p + i, 0, 0) << (8 * (i & 3));
      }
    }
  };

  f32x4_t acc[8][FN];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

  Scales sc, sc_next;
  load_scales(0, sc_next);
  static_for<0, NS>([&](auto T) {
    if (decltype(T)::value < kt_all) load_tile(decltype(T)::value, decltype(T)::value);
  });
  // waits until at most `tiles` of the newest tiles' loads are on their way
  auto wait_tiles = [&](int tiles) {
    if (NS > 3 && tiles >= 3) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * 3) : "memory");
    else if (NS > 2 && tiles == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * 2) : "memory");
    else if (tiles == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  wait_tiles(min(kt_all, NS) - 1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  Row ra0, ra1;  // the rows of two steps in turn
  i32x8_t fb[SUM == SUM_FP8 ? FN : 1];
  bf16x8g_t wb[SUM == SUM_F32 ? FN : 1][4];
  auto offset_b = [](int j) constexpr { return PAIR ? (j / RB) * 16 * RB * 128 + (j % RB) * 128 : j * 128; };
  auto widen_b = [&](auto J, const Row& r, const Scales& s) {
    constexpr int j = decltype(J)::value;
    const i32x8_t f = r.codes();
    if constexpr (SUM == SUM_FP8) {
      fb[j] = f;
    } else {
      const float e = SC == TP_GROUP_F32 ? 1.0f : e8m0_f32((s.eb >> (8 * j)) & 255);
#pragma unroll
      for (int c = 0; c < 4; ++c) wb[j][c] = widen<FMT_B>(f[2 * c], f[2 * c + 1], e);
    }
  };
  auto ask_a = [&](auto I, Row& r, int buf) {
    constexpr int i = decltype(I)::value;
    const uint32_t a0 = pa + buf * A_BYTES;
    if constexpr (SLDS) r.template ask<i * 128, i * 4>(a0, a0 ^ 16, ps + buf * S_BYTES);
    else r.template ask<i * 128>(a0, a0 ^ 16);
  };
  auto wait_a = [&](Row& r) {
    if constexpr (SLDS) r.wait_scale();
    else r.wait();
  };
  auto load_b = [&](int buf, const Scales& s) {  // the wavefront's columns of a tile
    const uint32_t b0 = pb + buf * B_BYTES;
    static_for<0, FN>([&](auto J) {
      Row r;
      r.template ask<offset_b(decltype(J)::value)>(b0, b0 ^ 16);
      r.wait();
      widen_b(J, r, s);
    });
  };

  f32x4_t p[FN];
  float sa = 0.0f;
  auto add_group = [&](auto I, auto J) {
    constexpr int i = decltype(I)::value, j = decltype(J)::value;
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(p[j][t], sa * sc.b[SQ ? 0 : t][j], acc[i][j][t]);
    asm volatile("" : "+v"(acc[i][j]));  // (put off past the barrier, it would hold its registers)
  };

  int buf = 0;
  sc = sc_next;
  load_b(0, sc);
  ask_a(std::integral_constant<int, 0>{}, ra0, 0);
  for (int kt = 0; kt < kt_all; ++kt) {
    const bool more = kt + 1 < kt_all;
    const int buf_next = buf + 1 == NS ? 0 : buf + 1;
    load_scales(more ? kt + 1 : kt, sc_next);
    static_for<0, 8>([&](auto I) {
      constexpr int i = decltype(I)::value;
      Row& r = i & 1 ? ra1 : ra0;
      Row& next = i & 1 ? ra0 : ra1;
      wait_a(r);
      if constexpr (i < 7) {
        ask_a(std::integral_constant<int, (i + 1) & 7>{}, next, buf);
      } else {
        // the tile is read; the next one is there for every wavefront after
        // this, and the buffer takes the one NS on
        wait_tiles(max(0, min(kt_all - 2 - kt, NS - 2)));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // (behind the last tile: rows that nothing uses, so that every path asks)
        ask_a(std::integral_constant<int, 0>{}, next, buf_next);
        if (kt + NS < kt_all) load_tile(kt + NS, buf);
      }
      const i32x8_t fa = r.codes();
      // fp32 scales: a step's group sums are scaled and added during the next
      // step, when the instructions that make them have ended
      if constexpr (SUM == SUM_F32) {
        float e = 1.0f;
        if constexpr (SC == TP_GROUP_E8M0) e = e8m0_f32((sc.ea[i >> 2] >> (8 * (i & 3))) & 255);
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
          __builtin_amdgcn_sched_barrier(0);
        });
      } else {
        static_for<0, FN>([&](auto J) {
          constexpr int j = decltype(J)::value;
          if constexpr (SC == TP_GROUP_F32) {
            if constexpr (i > 0) add_group(std::integral_constant<int, i - 1>{}, J);
            p[j] = mfma_plain<FMT_A, FMT_B>(fb[j], fa, (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f});
          } else {
            acc[i][j] = mfma_scaled<FMT_A, FMT_B, i & 3, j>(fb[j], fa, acc[i][j], (int)sc.eb, (int)sc.ea[i >> 2]);
          }
        });
      }
      if constexpr (SLDS) sa = r.s;
      if constexpr (SC == TP_GROUP_E8M0) {
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (SC == TP_GROUP_F32) {
      static_for<0, FN>([&](auto J) { add_group(std::integral_constant<int, 7>{}, J); });
    }
    sc = sc_next;
    load_b(buf_next, sc);
    buf = buf_next;
  }
  wait_a(ra0);
  __syncthreads();

  uint32_t* red = reinterpret_cast<uint32_t*>(lds);
  if constexpr (EPI == G_GLU_FWD) store_glu_fwd<WM, WN, FN, SC>(a, at, acc, red);
  else if constexpr (EPI == G_GLU_BWD) store_glu_bwd<WM, WN, FN, FMT_A, SC>(a, at, acc, red);
  else store_plain<WM, WN, FN>(a, at, acc);
}

template <int WM, int WN, int FN, int NS, int SC, bool SQ, int FMT_A, int FMT_B, int SUM, int EPI>
static hipError_t launch(G8GemmArgs& a, hipStream_t st) {
  constexpr int BM = 128 * WM, BN = EPI == G_GLU_FWD ? 8 * FN * WN : 16 * FN * WN;
  const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
  if (tm * tn > 0x7fffffff) return hipErrorInvalidValue;
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tn;
  if (tm * tn == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm<WM, WN, FN, NS, SC, SQ, FMT_A, FMT_B, SUM, EPI>), dim3((unsigned)(tm * tn)),
                     dim3(64 * WM * WN), 0, st, a);
  return hipGetLastError();
}

}  // namespace g8
}  // namespace tpmlp
