// extern "C" entry points of FP8 with group scales (include/tpmlp_fp8g.h):
// argument checks (host only), then launches on the caller's stream.
#include "checks.h"
#include "fp8g.h"

using namespace tpmlp;

namespace {

bool known_format(int f) { return f == TP_FP8_E4M3 || f == TP_FP8_E5M2; }
bool known_scale(int s) { return s == TP_GROUP_F32 || s == TP_GROUP_E8M0; }
size_t scale_bytes(int s) { return s == TP_GROUP_F32 ? 4 : 1; }

// scales: 4-byte aligned fp32 ones, bytes anywhere
int check_scales(int scale, const Buf* bufs, int n) {
  if (scale == TP_GROUP_F32) return check_tables(bufs, n);
  for (int i = 0; i < n; ++i)
    if (bufs[i].bytes && !bufs[i].p) return fail(TP_ERR_NULL, "%s is NULL", bufs[i].name);
  return TP_OK;
}

// codes and their scales: both there or neither
int check_pair(const void* q, const void* s, const char* qn, const char* sn) {
  if (!q == !s) return TP_OK;
  return fail(TP_ERR_NULL, "%s is NULL beside %s", q ? sn : qn, q ? qn : sn);
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(TP_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned16(ws)) return fail(TP_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (have < need) return fail(TP_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
  return TP_OK;
}

int check_glu(const tp_fp8g_glu_desc* d, bool backward) {
  if (!d) return fail(TP_ERR_NULL, "desc is NULL");
  if (d->gate != TP_GATE_SILU && d->gate != TP_GATE_GELU_TANH) return fail(TP_ERR_DTYPE, "unknown gate %d", d->gate);
  if (!known_scale(d->scale)) return fail(TP_ERR_DTYPE, "unknown scale %d", d->scale);
  if (!known_format(d->fmt) || (!backward && d->fmt != TP_FP8_E4M3)) return fail(TP_ERR_DTYPE, "unsupported format %d", d->fmt);
  if (d->N < 0 || d->N > kMaxDim) return fail(TP_ERR_SHAPE, "N out of range");
  if (d->H <= 0 || d->F <= 0 || d->H > kMaxLd || d->F > kMaxLd / 2) return fail(TP_ERR_SHAPE, "H or F out of range");
  if (d->H % 8 || d->F % 8) return fail(TP_ERR_SHAPE, "H and F must be multiples of 8");
  return TP_OK;
}

G8Form glu_form(const tp_fp8g_glu_desc& d, bool backward) {
  return g8_plan_glu(d.N, d.F, groups_of(d.H), backward);
}

// the fp32 values between the product and their quantization, where that is a
// launch of its own
size_t glu_workspace(const tp_fp8g_glu_desc& d, bool backward) {
  const G8Form form = glu_form(d, backward);
  const bool raw = form == G8_FEW || form == G8_SMALL;
  const size_t need = raw ? (size_t)d.N * (size_t)d.F * (backward ? 8 : 4) : 0;
  return need < 16 ? 16 : need;
}

}  // namespace

extern "C" {

int tp_fp8g_quantize(const tp_fp8g_quant_desc* desc, const void* x, void* q, void* s, void* q_t, void* s_t,
                     void* stream) {
  if (!desc) return fail(TP_ERR_NULL, "desc is NULL");
  const tp_fp8g_quant_desc& d = *desc;
  if (d.dtype != TP_F32 && d.dtype != TP_BF16) return fail(TP_ERR_DTYPE, "unknown dtype %d", d.dtype);
  if (!known_format(d.fmt)) return fail(TP_ERR_DTYPE, "unknown FP8 format %d", d.fmt);
  if (!known_scale(d.scale)) return fail(TP_ERR_DTYPE, "unknown scale %d", d.scale);
  if (d.square != 0 && d.square != 1) return fail(TP_ERR_SHAPE, "square must be 0 or 1");
  if (d.rows < 0 || d.rows > kMaxDim || d.cols <= 0 || d.cols > kMaxLd) return fail(TP_ERR_SHAPE, "rows or cols out of range");
  const int vec = d.dtype == TP_BF16 ? 8 : 4;
  if (d.cols % vec) return fail(TP_ERR_SHAPE, "cols must be a multiple of %d for this dtype", vec);
  int rc;
  if ((rc = check_pair(q, s, "q", "s")) || (rc = check_pair(q_t, s_t, "q_t", "s_t"))) return rc;
  if (!q && !q_t && d.rows > 0) return fail(TP_ERR_NULL, "q and q_t are NULL");
  const size_t e = scale_bytes(d.scale), rows = (size_t)d.rows, cols = (size_t)d.cols;
  const size_t gr = (size_t)groups_of(d.rows), gc = (size_t)groups_of(d.cols);
  Buf in[] = {{x, rows * cols * (d.dtype == TP_BF16 ? 2 : 4), "x"}};
  Buf codes[] = {{q, q ? rows * gc * kGroup : 0, "q"}, {q_t, q_t ? cols * gr * kGroup : 0, "q_t"}};
  Buf scales[] = {{s, s ? (d.square ? gr : rows) * gc * e : 0, "s"},
                  {s_t, s_t ? (d.square ? gc : cols) * gr * e : 0, "s_t"}};
  if ((rc = check_sized(in, 1)) || (rc = check_sized(codes, 2)) || (rc = check_scales(d.scale, scales, 2))) return rc;
  Buf outs[] = {codes[0], codes[1], scales[0], scales[1]};
  if ((rc = check_alias(in, 1, outs, 4)) || (rc = check_device())) return rc;
  G8QuantArgs a{x, (uint8_t*)q, (uint8_t*)q_t, s, s_t, d.rows, d.cols, d.cols, 1};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] { return g8_quant_launch(d.dtype, d.fmt, d.scale, d.square, a, st); });
  if (he != hipSuccess) return hip_fail(he, "group quantization launch");
  return ok();
}

int tp_fp8g_gemm(const tp_fp8g_gemm_desc* desc, const void* A, const void* sA, const void* B, const void* sB,
                 const void* B2, const void* sB2, void* C, void* stream) {
  if (!desc) return fail(TP_ERR_NULL, "desc is NULL");
  const tp_fp8g_gemm_desc& d = *desc;
  if (d.dtype != TP_F32 && d.dtype != TP_BF16) return fail(TP_ERR_DTYPE, "unknown dtype %d", d.dtype);
  if (!known_format(d.fmt_a) || !known_format(d.fmt_b) || (d.fmt_a == TP_FP8_E5M2 && d.fmt_b == TP_FP8_E5M2))
    return fail(TP_ERR_DTYPE, "unsupported FP8 formats %d, %d", d.fmt_a, d.fmt_b);
  if (!known_scale(d.scale)) return fail(TP_ERR_DTYPE, "unknown scale %d", d.scale);
  if (d.square != 0 && d.square != 1) return fail(TP_ERR_SHAPE, "square must be 0 or 1");
  if (d.accumulate != 0 && d.accumulate != 1) return fail(TP_ERR_SHAPE, "accumulate must be 0 or 1");
  if (d.accumulate && d.dtype != TP_F32) return fail(TP_ERR_DTYPE, "only fp32 is accumulated into");
  if (d.parts != 1 && d.parts != 2) return fail(TP_ERR_SHAPE, "parts must be 1 or 2");
  if (d.M < 0 || d.M > kMaxDim || d.N <= 0 || d.N > kMaxLd) return fail(TP_ERR_SHAPE, "M or N out of range");
  if (d.K < 0 || d.K > kMaxLd / d.parts || d.K % kGroup) return fail(TP_ERR_SHAPE, "K must be a multiple of 128 in range");
  // (the sum over an empty batch: a weight gradient, which is fp32)
  if (d.K == 0 && d.dtype != TP_F32) return fail(TP_ERR_SHAPE, "K must be positive for bf16 results");
  const int vec = d.dtype == TP_BF16 ? 8 : 4;
  if (d.N % vec) return fail(TP_ERR_SHAPE, "N must be a multiple of %d for this dtype", vec);
  const bool two = d.parts == 2;
  if (!two && (B2 || sB2)) return fail(TP_ERR_SHAPE, "B2 and sB2 must be NULL with one part");
  const size_t e = scale_bytes(d.scale), M = (size_t)d.M, N = (size_t)d.N, K = (size_t)d.K;
  const size_t nb = N * K, sb = (d.square ? (size_t)groups_of(d.N) : N) * (K / kGroup) * e;
  Buf codes[] = {{A, M * K * d.parts, "A"}, {B, nb, "B"}, {B2, two ? nb : 0, "B2"}};
  Buf scales[] = {{sA, M * (K / kGroup) * d.parts * e, "sA"}, {sB, sb, "sB"}, {sB2, two ? sb : 0, "sB2"}};
  Buf out[] = {{C, M * N * (d.dtype == TP_BF16 ? 2 : 4), "C"}};
  int rc;
  if ((rc = check_sized(codes, 3)) || (rc = check_sized(out, 1)) || (rc = check_scales(d.scale, scales, 3))) return rc;
  Buf ins[] = {codes[0], codes[1], codes[2], scales[0], scales[1], scales[2]};
  if ((rc = check_alias(ins, 6, out, 1)) || (rc = check_device())) return rc;
  G8GemmArgs a{};
  a.A = (const uint8_t*)A; a.B = (const uint8_t*)B; a.B2 = (const uint8_t*)B2;
  a.sA = sA; a.sB = sB; a.sB2 = sB2;
  a.M = d.M; a.lda = d.K * d.parts; a.N = (int)d.N; a.K = (int)d.K; a.parts = d.parts;
  a.C = C; a.out_bf16 = d.dtype == TP_BF16; a.accumulate = d.accumulate;
  if (d.M == 0 || (d.K == 0 && d.accumulate)) return ok();
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] {
    const bool f32 = !a.out_bf16, large = d.scale == TP_GROUP_E8M0 || d.square;
    // (of no groups FEW reads nothing and stores zeros)
    const G8Form form = d.K == 0 ? G8_FEW : g8_plan_gemm(d.M, d.N, d.K / kGroup * d.parts, f32, large);
    if (form == G8_FEW) return g8_gemm_few_launch(d.fmt_a, d.fmt_b, d.scale, d.square, a, st);
    return (f32 ? g8_gemm_f32_launch : g8_gemm_bf16_launch)(form == G8_LARGE, d.fmt_a, d.fmt_b, d.scale, d.square, a, st);
  });
  if (he != hipSuccess) return hip_fail(he, "group-scaled product launch");
  return ok();
}

size_t tp_fp8g_glu_fwd_workspace(const tp_fp8g_glu_desc* desc) {
  return check_glu(desc, false) ? 0 : glu_workspace(*desc, false);
}

int tp_fp8g_glu_fwd(const tp_fp8g_glu_desc* desc, const void* X, const void* sX, const void* Wg, const void* sWg,
                    const void* Wu, const void* sWu, void* Z_save, void* H_act, void* Hq, void* sH, void* Hq_t,
                    void* sH_t, void* workspace, size_t ws_bytes, void* stream) {
  if (int rc = check_glu(desc, false)) return rc;
  const tp_fp8g_glu_desc& d = *desc;
  int rc;
  if ((rc = check_pair(Hq, sH, "Hq", "sH")) || (rc = check_pair(Hq_t, sH_t, "Hq_t", "sH_t"))) return rc;
  if (!H_act && !Hq && !Hq_t && d.N > 0) return fail(TP_ERR_NULL, "H_act, Hq and Hq_t are NULL");
  const size_t e = scale_bytes(d.scale), N = (size_t)d.N, F = (size_t)d.F, ph = (size_t)padded(d.H);
  const size_t gh = ph / kGroup, gf = (size_t)groups_of(d.F), gn = (size_t)groups_of(d.N), need = glu_workspace(d, false);
  Buf in[] = {{X, N * ph, "X"}, {Wg, F * ph, "Wg"}, {Wu, F * ph, "Wu"}};
  Buf sin[] = {{sX, N * gh * e, "sX"}, {sWg, gf * gh * e, "sWg"}, {sWu, gf * gh * e, "sWu"}};
  Buf out[] = {{Z_save, Z_save ? N * 2 * F * 2 : 0, "Z_save"}, {H_act, H_act ? N * F * 2 : 0, "H_act"},
               {Hq, Hq ? N * gf * kGroup : 0, "Hq"}, {Hq_t, Hq_t ? F * gn * kGroup : 0, "Hq_t"}};
  Buf sout[] = {{sH, sH ? N * gf * e : 0, "sH"}, {sH_t, sH_t ? F * gn * e : 0, "sH_t"}};
  if ((rc = check_sized(in, 3)) || (rc = check_sized(out, 4)) || (rc = check_scales(d.scale, sin, 3)) ||
      (rc = check_scales(d.scale, sout, 2)) || (rc = check_ws(workspace, ws_bytes, need)))
    return rc;
  Buf ins[] = {in[0], in[1], in[2], sin[0], sin[1], sin[2]};
  Buf outs[] = {out[0], out[1], out[2], out[3], sout[0], sout[1], {workspace, need, "workspace"}};
  if ((rc = check_alias(ins, 6, outs, 7)) || (rc = check_device())) return rc;
  if (d.N == 0) return ok();
  G8GemmArgs a{};
  a.A = (const uint8_t*)X; a.B = (const uint8_t*)Wg; a.B2 = (const uint8_t*)Wu;
  a.sA = sX; a.sB = sWg; a.sB2 = sWu;
  a.M = d.N; a.lda = (int64_t)ph; a.N = (int)d.F; a.K = (int)ph; a.parts = 1;
  a.Z = Z_save; a.H = H_act; a.gate = d.gate;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] {
    const G8Form form = glu_form(d, false);
    if (form == G8_LARGE || form == G8_GROUP) {
      a.q = (uint8_t*)Hq; a.q_t = (uint8_t*)Hq_t; a.s = sH; a.s_t = sH_t;
      return g8_glu_fwd_launch(form, d.scale, a, st);
    }
    if (Hq || Hq_t) a.raw = (float*)workspace;
    hipError_t r = form == G8_FEW ? g8_glu_fwd_few_launch(d.scale, a, st) : g8_glu_fwd_launch(form, d.scale, a, st);
    if (r != hipSuccess || !a.raw) return r;
    const G8QuantArgs c{workspace, (uint8_t*)Hq, (uint8_t*)Hq_t, sH, sH_t, d.N, d.F, d.F, 1};
    return g8_quant_launch(TP_F32, TP_FP8_E4M3, d.scale, 0, c, st);
  });
  if (he != hipSuccess) return hip_fail(he, "gated block launch");
  return ok();
}

size_t tp_fp8g_glu_bwd_workspace(const tp_fp8g_glu_desc* desc) {
  return check_glu(desc, true) ? 0 : glu_workspace(*desc, true);
}

int tp_fp8g_glu_bwd(const tp_fp8g_glu_desc* desc, const void* dY, const void* sdY, const void* B, const void* sB,
                    const void* Z_save, void* dZ, void* sdZ, void* dZ_t, void* sdZ_t, void* workspace,
                    size_t ws_bytes, void* stream) {
  if (int rc = check_glu(desc, true)) return rc;
  const tp_fp8g_glu_desc& d = *desc;
  int rc;
  if ((rc = check_pair(dZ, sdZ, "dZ", "sdZ")) || (rc = check_pair(dZ_t, sdZ_t, "dZ_t", "sdZ_t"))) return rc;
  if (!dZ && !dZ_t && d.N > 0) return fail(TP_ERR_NULL, "dZ and dZ_t are NULL");
  const size_t e = scale_bytes(d.scale), N = (size_t)d.N, F = (size_t)d.F, ph = (size_t)padded(d.H);
  const size_t gh = ph / kGroup, gf = (size_t)groups_of(d.F), gn = (size_t)groups_of(d.N), need = glu_workspace(d, true);
  Buf in[] = {{dY, N * ph, "dY"}, {B, F * ph, "B"}, {Z_save, N * 2 * F * 2, "Z_save"}};
  Buf sin[] = {{sdY, N * gh * e, "sdY"}, {sB, gf * gh * e, "sB"}};
  Buf out[] = {{dZ, dZ ? N * 2 * gf * kGroup : 0, "dZ"}, {dZ_t, dZ_t ? 2 * F * gn * kGroup : 0, "dZ_t"}};
  Buf sout[] = {{sdZ, sdZ ? N * 2 * gf * e : 0, "sdZ"}, {sdZ_t, sdZ_t ? 2 * F * gn * e : 0, "sdZ_t"}};
  if ((rc = check_sized(in, 3)) || (rc = check_sized(out, 2)) || (rc = check_scales(d.scale, sin, 2)) ||
      (rc = check_scales(d.scale, sout, 2)) || (rc = check_ws(workspace, ws_bytes, need)))
    return rc;
  Buf ins[] = {in[0], in[1], in[2], sin[0], sin[1]};
  Buf outs[] = {out[0], out[1], sout[0], sout[1], {workspace, need, "workspace"}};
  if ((rc = check_alias(ins, 5, outs, 5)) || (rc = check_device())) return rc;
  if (d.N == 0) return ok();
  G8GemmArgs a{};
  a.A = (const uint8_t*)dY; a.B = (const uint8_t*)B;
  a.sA = sdY; a.sB = sB;
  a.M = d.N; a.lda = (int64_t)ph; a.N = (int)d.F; a.K = (int)ph; a.parts = 1;
  a.Z = const_cast<void*>(Z_save); a.gate = d.gate;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] {
    const G8Form form = glu_form(d, true);
    if (form == G8_LARGE || form == G8_GROUP) {
      a.q = (uint8_t*)dZ; a.q_t = (uint8_t*)dZ_t; a.s = sdZ; a.s_t = sdZ_t;
      return g8_glu_bwd_launch(form, d.fmt, d.scale, a, st);
    }
    a.raw = (float*)workspace;
    hipError_t r = form == G8_FEW ? g8_glu_bwd_few_launch(d.fmt, d.scale, a, st) : g8_glu_bwd_launch(form, d.fmt, d.scale, a, st);
    if (r != hipSuccess) return r;
    const G8QuantArgs c{workspace, (uint8_t*)dZ, (uint8_t*)dZ_t, sdZ, sdZ_t, d.N, d.F, 2 * d.F, 2};
    return g8_quant_launch(TP_F32, d.fmt, d.scale, 0, c, st);
  });
  if (he != hipSuccess) return hip_fail(he, "gated block backward launch");
  return ok();
}

}  // extern "C"
