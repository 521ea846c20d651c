// Host-side launchers of the operators around the products.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/tpmlp_block.h"

namespace tpmlp {

struct NormFwdArgs {
  const void *X, *O, *w_post, *b_post, *gate, *w_pre, *b_pre;
  void *Y, *Hn;
  float *stat_post, *stat_pre;
  int64_t N, G;  // G: gate rows, 0 without a gate
  int H;
  float eps, a, b;
};

struct NormBwdArgs {
  const void *dY, *dH, *Y, *O, *w_post, *b_post, *gate, *w_pre;
  const float *stat_post, *stat_pre;
  void *dX, *dO;
  float *dw_post, *db_post, *dgate, *dw_pre, *db_pre;
  float* ws;
  int64_t N, G;
  int H;
  int workers;  // rows are dealt to this many workers (see block_norm.hip)
  float a, b;
  int accumulate;
};

hipError_t norm_fwd_launch(int kind, int dtype, const NormFwdArgs& a, hipStream_t st);
hipError_t norm_bwd_launch(int kind, int dtype, NormBwdArgs& a, hipStream_t st);
size_t norm_bwd_workspace(const tp_norm_desc& d);

hipError_t route_fwd_launch(const tp_route_desc& d, const void* logits, const float* bias,
                            int32_t* expert, float* weight, hipStream_t st);
hipError_t route_bwd_launch(const tp_route_desc& d, const void* logits, const int32_t* expert,
                            const float* d_weight, const int32_t* slot_row, int64_t R,
                            void* dlogits, hipStream_t st);

struct TablesArgs {
  const int32_t* expert;
  const float* weight;
  int32_t *offsets, *row_token;
  float* row_weight;
  int32_t *tok_ptr, *tok_rows, *slot_row;
  int32_t* ws;
  int64_t N, R;
  int K, first, n_local;
};
size_t route_tables_workspace(int64_t N, int K, int n_local);
hipError_t route_tables_launch(const TablesArgs& a, hipStream_t st);

hipError_t adamw_launch(const tp_adamw_desc& d, int n, const tp_adamw_tensor* t,
                        const int32_t* dev_step, const float* dev_lr, const float* grad_scale,
                        hipStream_t st);

}  // namespace tpmlp
