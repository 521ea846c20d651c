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

// The 32 codes of a block's row that a lane has, waited for in the same
// place; with them, a row's scale
template <int OFF>
__device__ __forceinline__ i32x8_t read_codes(uint32_t a0, uint32_t a1) {
  i32x4_t lo, hi;
  asm volatile("ds_read_b128 %0, %2 offset:%4\n\tds_read_b128 %1, %3 offset:%4\n\ts_waitcnt lgkmcnt(0)"
               : "=&v"(lo), "=&v"(hi) : "v"(a0), "v"(a1), "n"(OFF) : "memory");
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int OFF, int SOFF>
__device__ __forceinline__ i32x8_t read_codes_scale(uint32_t a0, uint32_t a1, uint32_t as, float& s) {
  i32x4_t lo, hi;
  asm volatile("ds_read_b128 %0, %3 offset:%6\n\tds_read_b128 %1, %4 offset:%6\n\tds_read_b32 %2, %5 offset:%7\n\t"
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(lo), "=&v"(hi), "=&v"(s) : "v"(a0), "v"(a1), "v"(as), "n"(OFF), "n"(SOFF) : "memory");
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

struct __attribute__((packed)) Bytes8 { uint32_t v[2]; };

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
  const uint32_t c0 = ((2 * at.q) ^ (at.p & 7)) << 4, c1 = c0 ^ 16;
  uint32_t pa = l0 + (at.wm * 128 + 8 * at.p) * 128, pb = l0 + B_AT + (at.wn * 16 * FN + at.p * RB) * 128;
  uint32_t ps = l0 + S_AT + (at.wm * 128 + 8 * at.p) * 4;

  // column of index b of block j, and its scale's place
  auto col_of = [&](int b, int j) -> int64_t {
    return PAIR ? at.n0 + at.wn * 8 * FN + b * RB + j % RB : at.n0 + at.wn * 16 * FN + b * FN + j;
  };
  const int64_t mr = at.m0 + 8 * at.p;
  const bool whole = at.m0 + 128 <= a.M;  // every row of the wavefront is there

  f32x4_t acc[8][FN];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f};

  static_for<0, NS>([&](auto T) {
    if (decltype(T)::value < kt_all) load_tile(decltype(T)::value, decltype(T)::value);
  });
  int buf = 0;
  for (int kt = 0; kt < kt_all; ++kt) {
    const int part = kt >= kt_part ? 1 : 0, kb = kt - part * kt_part;
    auto sb_src = [&](int j) { return PAIR ? (j < FN / 2 ? a.sB : a.sB2) : (part ? a.sB2 : a.sB); };
    auto scale_b = [&](int b, int j) {
      const int64_t n = min(col_of(b, j), (int64_t)a.N - 1);
      return SQ ? n / kGroup * kt_part + kb : (int64_t)kb * a.N + n;
    };
    // column scales (and E8M0 row scales) of this tile
    constexpr int SBT = SC == TP_GROUP_F32 && !SQ ? 4 : 1;
    float sb[SBT][FN];
    uint32_t eb = 0, ea[2] = {0, 0};
    if constexpr (SC == TP_GROUP_F32) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int t = 0; t < SBT; ++t)
          sb[t][j] = reinterpret_cast<const float*>(sb_src(j))[scale_b(SQ ? 0 : 4 * at.q + t, j)];
    } else {
#pragma unroll
      for (int j = 0; j < FN; ++j) eb |= (uint32_t)reinterpret_cast<const uint8_t*>(sb_src(j))[scale_b(SQ ? 0 : at.p, j)] << (8 * j);
      const uint8_t* s = reinterpret_cast<const uint8_t*>(a.sA) + (int64_t)kt * a.M;
      if (whole) {
        const Bytes8 w = *reinterpret_cast<const Bytes8*>(s + mr);
        ea[0] = w.v[0];
        ea[1] = w.v[1];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) ea[i >> 2] |= (uint32_t)s[min(mr + i, a.M - 1)] << (8 * (i & 3));
      }
    }
    // this tile is there; the next ones' loads may still be on their way
    const int ahead = kt_all - 1 - kt;
    if (ahead >= NS - 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * (NS - 1)) : "memory");
    else if (NS > 3 && ahead == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS * 2) : "memory");
    else if (NS > 2 && ahead == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    const uint32_t a0 = pa + buf * A_BYTES + c0, a1 = pa + buf * A_BYTES + c1, as = ps + buf * S_BYTES;
    const uint32_t b0 = pb + buf * B_BYTES + c0, b1 = pb + buf * B_BYTES + c1;
    i32x8_t fb[FN];
    bf16x8g_t wb[SUM == SUM_F32 ? FN : 1][4];
    static_for<0, FN>([&](auto J) {
      constexpr int j = decltype(J)::value;
      fb[j] = read_codes<PAIR ? (j / RB) * 16 * RB * 128 + (j % RB) * 128 : j * 128>(b0, b1);
      if constexpr (SUM == SUM_F32) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          wb[j][c] = widen<FMT_B>(fb[j][2 * c], fb[j][2 * c + 1], SC == TP_GROUP_F32 ? 1.0f : e8m0_f32((eb >> (8 * j)) & 255));
      }
    });
    static_for<0, 8>([&](auto I) {
      constexpr int i = decltype(I)::value;
      float sa = 1.0f;
      i32x8_t fa;
      if constexpr (SLDS) fa = read_codes_scale<i * 128, i * 4>(a0, a1, as, sa);
      else fa = read_codes<i * 128>(a0, a1);
      if constexpr (SUM == SUM_F32) {
        if constexpr (SC == TP_GROUP_E8M0) sa = e8m0_f32((ea[i >> 2] >> (8 * (i & 3))) & 255);
        f32x4_t p[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) p[j] = SC == TP_GROUP_F32 ? (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bf16x8g_t wa = widen<FMT_A>(fa[2 * c], fa[2 * c + 1], SC == TP_GROUP_F32 ? 1.0f : sa);
#pragma unroll
          for (int j = 0; j < FN; ++j) p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][c], wa, p[j], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (SC == TP_GROUP_F32) {
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(p[j][t], sa * sb[SQ ? 0 : t][j], acc[i][j][t]);
          } else {
            acc[i][j] = p[j];
          }
        }
      } else if constexpr (SC == TP_GROUP_F32) {
        f32x4_t p[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) p[j] = mfma_plain<FMT_A, FMT_B>(fb[j], fa, (f32x4_t){0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[i][j][t] = fmaf(p[j][t], sa * sb[SQ ? 0 : t][j], acc[i][j][t]);
      } else {
        static_for<0, FN>([&](auto J) {
          constexpr int j = decltype(J)::value;
          acc[i][j] = mfma_scaled<FMT_A, FMT_B, i & 3, j>(fb[j], fa, acc[i][j], (int)eb, (int)ea[i >> 2]);
        });
      }
      // (the reads of later rows moved up, or these sums put off past the
      // barrier, would need registers of their own)
#pragma unroll
      for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
      __builtin_amdgcn_sched_barrier(0);
    });
    // every wavefront has read this tile: its buffer takes the one NS on
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (kt + NS < kt_all) load_tile(kt + NS, buf);
    buf = buf + 1 == NS ? 0 : buf + 1;
  }

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
