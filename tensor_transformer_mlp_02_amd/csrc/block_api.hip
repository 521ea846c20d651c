// extern "C" entry points of the operators around the products
// (include/tpmlp_block.h): argument checks (host only), then launches on
// the caller's stream.
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "block_launch.h"
#include "checks.h"

using namespace tpmlp;

namespace {

int check_norm(const tp_norm_desc* d) {
  if (!d) return fail(TP_ERR_NULL, "desc is NULL");
  if (d->dtype != TP_F32 && d->dtype != TP_BF16)
    return fail(TP_ERR_DTYPE, "unknown dtype %d", d->dtype);
  if (d->kind != TP_NORM_RMS && d->kind != TP_NORM_LAYER)
    return fail(TP_ERR_DTYPE, "unknown norm %d", d->kind);
  if (d->N < 0 || d->H <= 0 || d->gate_rows < 0)
    return fail(TP_ERR_SHAPE, "N and gate_rows must be >= 0 and H > 0");
  if (d->N > kMaxDim || d->H > kMaxLd || d->gate_rows > kMaxDim)
    return fail(TP_ERR_SHAPE, "dimension too large");
  const int vec = d->dtype == TP_BF16 ? 8 : 4;
  if (d->H % vec) return fail(TP_ERR_SHAPE, "H must be a multiple of %d for this dtype", vec);
  if (!(d->eps > 0.f) || !isfinite(d->eps)) return fail(TP_ERR_SHAPE, "eps must be positive and finite");
  if (!isfinite(d->res_scale) || !isfinite(d->branch_scale))
    return fail(TP_ERR_SHAPE, "res_scale and branch_scale must be finite");
  return TP_OK;
}

// a buffer that must be there exactly when `wanted`
int check_wanted(const void* p, bool wanted, const char* name, const char* why) {
  if (wanted && !p) return fail(TP_ERR_NULL, "%s is NULL", name);
  if (!wanted && p) return fail(TP_ERR_SHAPE, "%s must be NULL %s", name, why);
  return TP_OK;
}

int check_route(const tp_route_desc* d) {
  if (!d) return fail(TP_ERR_NULL, "desc is NULL");
  if (d->dtype != TP_F32 && d->dtype != TP_BF16)
    return fail(TP_ERR_DTYPE, "unknown dtype %d", d->dtype);
  if (d->score != TP_SCORE_SOFTMAX && d->score != TP_SCORE_SIGMOID)
    return fail(TP_ERR_DTYPE, "unknown score %d", d->score);
  if (d->E < 1 || d->E > TP_ROUTE_MAX_EXPERTS)
    return fail(TP_ERR_SHAPE, "E must be in 1..%d", TP_ROUTE_MAX_EXPERTS);
  if (d->groups < 1 || d->groups > TP_ROUTE_MAX_GROUPS || d->E % d->groups)
    return fail(TP_ERR_SHAPE, "groups must be in 1..%d and divide E", TP_ROUTE_MAX_GROUPS);
  if (d->groups_kept < 1 || d->groups_kept > d->groups)
    return fail(TP_ERR_SHAPE, "groups_kept must be in 1..groups");
  if (d->group_best != 1 && d->group_best != 2)
    return fail(TP_ERR_SHAPE, "group_best must be 1 or 2");
  if (d->K < 1 || d->K > TP_ROUTE_MAX_K || d->K > d->groups_kept * (d->E / d->groups))
    return fail(TP_ERR_SHAPE, "K must be in 1..%d and at most the experts of the groups kept",
                TP_ROUTE_MAX_K);
  if (d->renorm != 0 && d->renorm != 1) return fail(TP_ERR_SHAPE, "renorm must be 0 or 1");
  if (!isfinite(d->scale)) return fail(TP_ERR_SHAPE, "scale must be finite");
  if (d->N < 0 || d->N > kMaxDim || d->N * d->E >= ((int64_t)1 << 40))
    return fail(TP_ERR_SHAPE, "N out of range");
  return TP_OK;
}

int check_tables_shape(int64_t N, int32_t K, int32_t n_local) {
  if (K < 1 || K > TP_ROUTE_MAX_K) return fail(TP_ERR_SHAPE, "K must be in 1..%d", TP_ROUTE_MAX_K);
  if (n_local < 1 || n_local > TP_ROUTE_MAX_EXPERTS)
    return fail(TP_ERR_SHAPE, "n_local must be in 1..%d", TP_ROUTE_MAX_EXPERTS);
  if (N < 0 || N > kMaxDim || N * K > 0x7fffffff)
    return fail(TP_ERR_SHAPE, "N out of range (N*K below 2^31)");
  return TP_OK;
}

// The step's buffers, to see that no two overlap.  Those of one kind usually
// lie in the list's order: then each has to start behind the one before and
// the kinds have to lie apart as wholes, told in one walk; otherwise they are
// all sorted.
struct Span {
  uintptr_t lo, hi;
  int32_t tensor;
  const char* name;
};
struct Kind {
  uintptr_t lo = 0, hi = 0;
  bool ordered = true;
  void add(const Buf& b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(b.p);
    if (!hi) lo = p;
    else if (p < hi) ordered = false;
    hi = p + b.bytes;
  }
};

constexpr int kKinds = 7;
void step_buffers(const tp_adamw_tensor& t, size_t ge, size_t se, bool q, Buf (&b)[kKinds]) {
  const size_t c = (size_t)t.count, blocks = (c + TP_ADAMW_BLOCK - 1) / TP_ADAMW_BLOCK;
  b[0] = {t.param, c * 4, "param"};
  b[1] = {t.grad, c * ge, "grad"};
  b[2] = {t.m, c * se, "m"};
  b[3] = {t.v, c * se, "v"};
  b[4] = {t.param_bf16, t.param_bf16 ? c * 2 : 0, "param_bf16"};
  b[5] = {t.m_scale, q ? blocks * 4 : 0, "m_scale"};
  b[6] = {t.v_scale, q ? blocks * 4 : 0, "v_scale"};
}

}  // namespace

extern "C" {

int tp_block_norm_fwd(const tp_norm_desc* desc, const void* X, const void* O, const void* w_post,
                      const void* b_post, const void* gate, const void* w_pre, const void* b_pre,
                      void* Y, void* Hn, float* stat_post, float* stat_pre, void* stream) {
  if (int rc = check_norm(desc)) return rc;
  const tp_norm_desc& d = *desc;
  const size_t e = d.dtype == TP_BF16 ? 2 : 4;
  const size_t rows = (size_t)(d.N * d.H) * e, vec = (size_t)d.H * e;
  const size_t stat = (size_t)d.N * 4 * (d.kind == TP_NORM_LAYER ? 2 : 1);
  // (without tokens every row buffer may be NULL: nothing tells a block's absence)
  if (!O && d.N > 0 && (w_post || b_post || gate || d.gate_rows || Y || stat_post))
    return fail(TP_ERR_SHAPE, "w_post, b_post, gate, Y and stat_post need O");
  if (b_post && !w_post) return fail(TP_ERR_NULL, "w_post is NULL");
  if (b_pre && !w_pre) return fail(TP_ERR_NULL, "w_pre is NULL");
  if (!O && d.N > 0 && !w_pre) return fail(TP_ERR_NULL, "w_pre is NULL");
  int rc;
  if ((rc = check_wanted(gate, d.gate_rows > 0, "gate", "with gate_rows 0"))) return rc;
  if (stat_post && !w_post) return fail(TP_ERR_SHAPE, "stat_post must be NULL without w_post");
  if (stat_pre && !w_pre) return fail(TP_ERR_SHAPE, "stat_pre must be NULL without w_pre");
  if (!w_pre && Hn) return fail(TP_ERR_SHAPE, "Hn must be NULL without w_pre");
  Buf ins[] = {{X, rows, "X"},
               {O, O ? rows : 0, "O"},
               {w_post, w_post ? vec : 0, "w_post"},
               {b_post, b_post ? vec : 0, "b_post"},
               {gate, (size_t)d.gate_rows * vec, "gate"},
               {w_pre, w_pre ? vec : 0, "w_pre"},
               {b_pre, b_pre ? vec : 0, "b_pre"}};
  Buf outs[] = {{Y, O ? rows : 0, "Y"}, {Hn, w_pre ? rows : 0, "Hn"}};
  Buf stats[] = {{stat_post, stat_post ? stat : 0, "stat_post"},
                 {stat_pre, stat_pre ? stat : 0, "stat_pre"}};
  if ((rc = check_sized(ins, 7)) || (rc = check_sized(outs, 2)) || (rc = check_tables(stats, 2)))
    return rc;
  // Y may be X itself
  Buf apart[] = {{Y == X ? nullptr : X, rows, "X"}, ins[1], ins[2], ins[3], ins[4], ins[5], ins[6]};
  Buf all[] = {outs[0], outs[1], stats[0], stats[1]};
  if ((rc = check_alias(apart, 7, all, 4))) return rc;
  if ((rc = check_device())) return rc;
  NormFwdArgs a{X, O, w_post, b_post, gate, w_pre, b_pre, Y, Hn, stat_post, stat_pre,
                d.N, d.gate_rows, (int)d.H, d.eps, d.res_scale, d.branch_scale};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] { return norm_fwd_launch(d.kind, d.dtype, a, st); });
  if (he != hipSuccess) return hip_fail(he, "block norm launch");
  return ok();
}

size_t tp_block_norm_bwd_workspace(const tp_norm_desc* desc) {
  if (check_norm(desc)) return 0;
  return norm_bwd_workspace(*desc);
}

int tp_block_norm_bwd(const tp_norm_desc* desc, const void* dY, const void* dHn, const void* Y,
                      const void* O, const void* w_post, const void* b_post, const void* gate,
                      const void* w_pre, const float* stat_post, const float* stat_pre, void* dX,
                      void* dO, float* dw_post, float* db_post, float* dgate, float* dw_pre,
                      float* db_pre, void* workspace, size_t ws_bytes, int32_t accumulate,
                      void* stream) {
  if (int rc = check_norm(desc)) return rc;
  const tp_norm_desc& d = *desc;
  const size_t e = d.dtype == TP_BF16 ? 2 : 4;
  const size_t rows = (size_t)(d.N * d.H) * e, vec = (size_t)d.H * e, out = (size_t)d.H * 4;
  const size_t stat = (size_t)d.N * 4 * (d.kind == TP_NORM_LAYER ? 2 : 1);
  int rc;
  if (accumulate != 0 && accumulate != 1) return fail(TP_ERR_SHAPE, "accumulate must be 0 or 1");
  // (without tokens every row buffer may be NULL: nothing tells a block's absence)
  if (!O && d.N > 0 && (w_post || b_post || gate || d.gate_rows || dO || stat_post || dw_post || db_post || dgate))
    return fail(TP_ERR_SHAPE, "w_post, b_post, gate and their gradients need O");
  if (!O && d.N > 0 && !w_pre) return fail(TP_ERR_NULL, "w_pre is NULL");
  if (b_post && !w_post) return fail(TP_ERR_NULL, "w_post is NULL");
  if ((rc = check_wanted(dw_post, w_post != nullptr, "dw_post", "without w_post"))) return rc;
  if (db_post && !w_post) return fail(TP_ERR_SHAPE, "db_post must be NULL without w_post");
  if ((rc = check_wanted(dw_pre, w_pre != nullptr, "dw_pre", "without w_pre"))) return rc;
  if (db_pre && !w_pre) return fail(TP_ERR_SHAPE, "db_pre must be NULL without w_pre");
  if (!w_pre && dHn) return fail(TP_ERR_SHAPE, "dHn must be NULL without w_pre");
  if (!w_pre && d.N > 0 && !dY) return fail(TP_ERR_NULL, "dY is NULL");
  if ((rc = check_wanted(gate, d.gate_rows > 0, "gate", "with gate_rows 0"))) return rc;
  if ((rc = check_wanted(dgate, d.gate_rows > 0, "dgate", "with gate_rows 0"))) return rc;
  const size_t need = norm_bwd_workspace(d);
  if (!workspace) return fail(TP_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if (!aligned16(workspace)) return fail(TP_ERR_ALIGN, "workspace is not 16-byte aligned");
  if (ws_bytes < need)
    return fail(TP_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, need);
  Buf ins[] = {{dY, dY ? rows : 0, "dY"},
               {dHn, w_pre ? rows : 0, "dHn"},
               {Y, w_pre ? rows : 0, "Y"},
               {O, O ? rows : 0, "O"},
               {w_post, w_post ? vec : 0, "w_post"},
               {b_post, b_post ? vec : 0, "b_post"},
               {gate, (size_t)d.gate_rows * vec, "gate"},
               {w_pre, w_pre ? vec : 0, "w_pre"},
               {stat_post, w_post ? stat : 0, "stat_post"},
               {stat_pre, w_pre ? stat : 0, "stat_pre"}};
  Buf outs[] = {{dX, rows, "dX"},
                {dO, O ? rows : 0, "dO"},
                {dw_post, w_post ? out : 0, "dw_post"},
                {db_post, db_post ? out : 0, "db_post"},
                {dgate, (size_t)d.gate_rows * out, "dgate"},
                {dw_pre, w_pre ? out : 0, "dw_pre"},
                {db_pre, db_pre ? out : 0, "db_pre"},
                {workspace, need, "workspace"}};
  if ((rc = check_sized(ins, 8)) || (rc = check_tables(ins + 8, 2)) || (rc = check_sized(outs, 7)))
    return rc;
  if ((rc = check_alias(ins, 10, outs, 8))) return rc;
  if ((rc = check_device())) return rc;
  NormBwdArgs a{dY, dHn, Y, O, w_post, b_post, gate, w_pre, stat_post, stat_pre, dX, dO,
                dw_post, db_post, dgate, dw_pre, db_pre, reinterpret_cast<float*>(workspace),
                d.N, d.gate_rows, (int)d.H, 0, d.res_scale, d.branch_scale, accumulate};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] { return norm_bwd_launch(d.kind, d.dtype, a, st); });
  if (he != hipSuccess) return hip_fail(he, "block norm backward launch");
  return ok();
}

int tp_moe_route_fwd(const tp_route_desc* desc, const void* logits, const float* bias,
                     int32_t* topk_expert, float* topk_weight, void* stream) {
  if (int rc = check_route(desc)) return rc;
  const tp_route_desc& d = *desc;
  const size_t e = d.dtype == TP_BF16 ? 2 : 4;
  Buf in[] = {{logits, (size_t)(d.N * d.E) * e, "logits"}};
  Buf tab[] = {{bias, bias ? (size_t)d.E * 4 : 0, "bias"},
               {topk_expert, (size_t)(d.N * d.K) * 4, "topk_expert"},
               {topk_weight, (size_t)(d.N * d.K) * 4, "topk_weight"}};
  if (int rc = check_sized(in, 1)) return rc;
  if (int rc = check_tables(tab, 3)) return rc;
  Buf ins[] = {in[0], tab[0]};
  if (int rc = check_alias(ins, 2, tab + 1, 2)) return rc;
  if (int rc = check_device()) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] {
    return route_fwd_launch(d, logits, bias, topk_expert, topk_weight, st);
  });
  if (he != hipSuccess) return hip_fail(he, "routing launch");
  return ok();
}

int tp_moe_route_bwd(const tp_route_desc* desc, const void* logits, const int32_t* topk_expert,
                     const float* d_weight, const int32_t* slot_row, int64_t R, void* dlogits,
                     void* stream) {
  if (int rc = check_route(desc)) return rc;
  const tp_route_desc& d = *desc;
  if (R < 0 || R > ((int64_t)1 << 40)) return fail(TP_ERR_SHAPE, "R out of range");
  const size_t e = d.dtype == TP_BF16 ? 2 : 4;
  const size_t slots = (size_t)(d.N * d.K) * 4;
  Buf in[] = {{logits, (size_t)(d.N * d.E) * e, "logits"}};
  Buf out[] = {{dlogits, (size_t)(d.N * d.E) * e, "dlogits"}};
  Buf tab[] = {{topk_expert, slots, "topk_expert"},
               {d_weight, slot_row ? (d.N > 0 ? (size_t)R * 4 : 0) : slots, "d_weight"},
               {slot_row, slot_row ? slots : 0, "slot_row"}};
  if (int rc = check_sized(in, 1)) return rc;
  if (int rc = check_sized(out, 1)) return rc;
  if (int rc = check_tables(tab, 3)) return rc;
  Buf ins[] = {in[0], tab[0], tab[1], tab[2]};
  if (int rc = check_alias(ins, 4, out, 1)) return rc;
  if (int rc = check_device()) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] {
    return route_bwd_launch(d, logits, topk_expert, d_weight, slot_row, R, dlogits, st);
  });
  if (he != hipSuccess) return hip_fail(he, "routing backward launch");
  return ok();
}

size_t tp_moe_route_tables_workspace(int64_t N, int32_t K, int32_t n_local) {
  if (check_tables_shape(N, K, n_local)) return 0;
  return route_tables_workspace(N, K, n_local);
}

int tp_moe_route_tables(int64_t N, int32_t K, int32_t first_expert, int32_t n_local, int64_t R,
                        const int32_t* topk_expert, const float* topk_weight, int32_t* offsets,
                        int32_t* row_token, float* row_weight, int32_t* tok_ptr,
                        int32_t* tok_rows, int32_t* slot_row, void* workspace, size_t ws_bytes,
                        void* stream) {
  if (int rc = check_tables_shape(N, K, n_local)) return rc;
  if (first_expert < 0) return fail(TP_ERR_SHAPE, "first_expert must be >= 0");
  if (R < N * K || R > 0x7fffffff)
    return fail(TP_ERR_SHAPE, "R must be in N*K .. 2^31-1 (every choice may be local)");
  if ((topk_weight != nullptr || N == 0) != (row_weight != nullptr || R == 0) && N > 0)
    return fail(TP_ERR_NULL, "topk_weight and row_weight come together");
  const size_t need = route_tables_workspace(N, K, n_local);
  if (need > 0) {
    if (!workspace) return fail(TP_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (!aligned16(workspace)) return fail(TP_ERR_ALIGN, "workspace is not 16-byte aligned");
    if (ws_bytes < need)
      return fail(TP_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, need);
  }
  const size_t slots = (size_t)(N * K) * 4, rb = (size_t)R * 4;
  Buf ins[] = {{topk_expert, slots, "topk_expert"},
               {topk_weight, topk_weight ? slots : 0, "topk_weight"}};
  Buf outs[] = {{offsets, ((size_t)n_local + 1) * 4, "offsets"},
                {row_token, rb, "row_token"},
                {row_weight, row_weight ? rb : 0, "row_weight"},
                {tok_ptr, ((size_t)N + 1) * 4, "tok_ptr"},
                {tok_rows, rb, "tok_rows"},
                {slot_row, slots, "slot_row"},
                {workspace, need, "workspace"}};
  if (int rc = check_tables(ins, 2)) return rc;
  if (int rc = check_tables(outs, 6)) return rc;
  if (int rc = check_alias(ins, 2, outs, 7)) return rc;
  if (int rc = check_device()) return rc;
  TablesArgs a{topk_expert, topk_weight, offsets, row_token, row_weight, tok_ptr, tok_rows,
               slot_row, reinterpret_cast<int32_t*>(workspace), N, R, K, first_expert, n_local};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] { return route_tables_launch(a, st); });
  if (he != hipSuccess) return hip_fail(he, "dispatch tables launch");
  return ok();
}

int tp_adamw_step(const tp_adamw_desc* desc, int32_t n, const tp_adamw_tensor* tensors,
                  const int32_t* dev_step, const float* dev_lr, const float* grad_scale,
                  void* stream) {
  if (!desc) return fail(TP_ERR_NULL, "desc is NULL");
  const tp_adamw_desc& d = *desc;
  if (d.grad_dtype != TP_F32 && d.grad_dtype != TP_BF16)
    return fail(TP_ERR_DTYPE, "unknown grad_dtype %d", d.grad_dtype);
  if (d.state_bits != 32 && d.state_bits != 8)
    return fail(TP_ERR_DTYPE, "state_bits must be 32 or 8");
  if (!isfinite((float)d.lr)) return fail(TP_ERR_SHAPE, "lr must be finite in fp32");
  if (!(d.beta1 >= 0.0 && d.beta1 < 1.0) || !(d.beta2 >= 0.0 && d.beta2 < 1.0))
    return fail(TP_ERR_SHAPE, "beta1 and beta2 must be in [0, 1)");
  // eps keeps its meaning in fp32
  if (!(d.eps >= 1e-30 && d.eps <= 1e30)) return fail(TP_ERR_SHAPE, "eps must be in 1e-30..1e30");
  if (!dev_step && d.step < 1) return fail(TP_ERR_SHAPE, "step counts from 1");
  if (n < 0 || n > TP_ADAMW_MAX_TENSORS)
    return fail(TP_ERR_SHAPE, "n must be in 0..%d", TP_ADAMW_MAX_TENSORS);
  if (n > 0 && !tensors) return fail(TP_ERR_NULL, "tensors is NULL");
  if ((reinterpret_cast<uintptr_t>(dev_step) | reinterpret_cast<uintptr_t>(dev_lr) |
       reinterpret_cast<uintptr_t>(grad_scale)) & 3u)
    return fail(TP_ERR_ALIGN, "dev_step, dev_lr and grad_scale must be 4-byte aligned");
  const bool q = d.state_bits == 8;
  const size_t ge = d.grad_dtype == TP_BF16 ? 2 : 4, se = q ? 1 : 4;
  int rc;
  Kind kinds[kKinds];
  Buf b[kKinds];
  for (int32_t i = 0; i < n; ++i) {
    const tp_adamw_tensor& t = tensors[i];
    if (t.count < 0 || t.count > ((int64_t)1 << 40))
      return fail(TP_ERR_SHAPE, "count of tensor %d must be in 0..2^40", i);
    if (!isfinite(t.weight_decay))
      return fail(TP_ERR_SHAPE, "weight_decay of tensor %d must be finite", i);
    if (t.reserved != 0) return fail(TP_ERR_SHAPE, "reserved of tensor %d must be 0", i);
    if (!q && (t.m_scale || t.v_scale))
      return fail(TP_ERR_SHAPE, "m_scale and v_scale of tensor %d must be NULL with 32-bit states", i);
    step_buffers(t, ge, se, q, b);
    if ((rc = check_sized(b, 5)) || (rc = check_tables(b + 5, 2))) return rc;
    for (int k = 0; k < kKinds; ++k)
      if (b[k].bytes > 0) kinds[k].add(b[k]);
  }
  bool apart = true;
  for (int k = 0; k < kKinds; ++k) {
    apart = apart && kinds[k].ordered;
    for (int j = 0; j < k; ++j)
      if (kinds[k].hi && kinds[j].hi)
        apart = apart && (kinds[k].hi <= kinds[j].lo || kinds[j].hi <= kinds[k].lo);
  }
  // the device scalars are read throughout the step
  const void* scalars[] = {dev_step, dev_lr, grad_scale};
  for (const void* p : scalars)
    for (int k = 0; p && k < kKinds; ++k) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      if (kinds[k].hi && lo < kinds[k].hi && kinds[k].lo < lo + 4) apart = false;
    }
  if (!apart) {
    try {
      std::vector<Span> all;
      all.reserve((size_t)n * kKinds + 3);
      for (int32_t i = 0; i < n; ++i) {
        step_buffers(tensors[i], ge, se, q, b);
        for (int k = 0; k < kKinds; ++k) {
          const uintptr_t lo = reinterpret_cast<uintptr_t>(b[k].p);
          if (b[k].bytes > 0) all.push_back(Span{lo, lo + b[k].bytes, i, b[k].name});
        }
      }
      std::sort(all.begin(), all.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
      for (size_t i = 1; i < all.size(); ++i)
        if (all[i].lo < all[i - 1].hi)
          return fail(TP_ERR_ALIAS, "%s of tensor %d and %s of tensor %d overlap", all[i - 1].name,
                      all[i - 1].tensor, all[i].name, all[i].tensor);
      for (const void* p : scalars) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        for (const Span& x : all)
          if (p && lo < x.hi && x.lo < lo + 4)
            return fail(TP_ERR_ALIAS, "a device scalar lies in %s of tensor %d", x.name, x.tensor);
      }
    } catch (const std::bad_alloc&) {
      return fail(TP_ERR_SHAPE, "out of host memory for %d tensors", n);
    }
  }
  if ((rc = check_device())) return rc;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipError_t he = timed(st, [&] {
    return adamw_launch(d, n, tensors, dev_step, dev_lr, grad_scale, st);
  });
  if (he != hipSuccess) return hip_fail(he, "AdamW launch");
  return ok();
}

}  // extern "C"
