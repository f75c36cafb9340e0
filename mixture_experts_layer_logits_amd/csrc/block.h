// Internal declarations: the operators around the expert layer (router balance loss, block
// norms with gate and residual scale, and the combine fused with them).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include "common.h"

namespace moe {

// ------------------------------------------------------------------ balance loss
constexpr int kBalanceBlocks = 256;  // most workgroups (rows of partial sums) of the forward
size_t balance_workspace_bytes(int T, int E, int k);
hipError_t balance_forward(int T, int E, int k, const float* logits, const int32_t* topk_idx, const uint8_t* mask,
                           float* lse, int32_t* counts, float* prob_mean, float* loss, void* ws, hipStream_t st);
hipError_t balance_backward(int T, int E, int k, const float* logits, const float* lse, const int32_t* counts,
                            const float* dloss, const float* dgates, const float* gates, const int32_t* topk_idx,
                            float* dlogits, hipStream_t st);

// ------------------------------------------------------------------ block norms
constexpr int kNormMaxWidth = 16384;  // widest row the kernels hold in registers
constexpr int kNormBlocks = 512;      // most workgroups (rows of weight-gradient partials) of the backward

// Pointers of one call; elem: float or bf16 rows and norm weights (all [T][d] or [d]), the rest
// as typed.  y_perm != nullptr: the branch is the gated sum of k routed rows (+ y_add) instead
// of y.
struct NormFwd {
  int T, d, k;
  const void *x, *y, *y_perm, *y_add, *w_post, *w_pre;
  const float *gates, *gate;
  const int32_t* slot_row;
  float res_scale, eps;
  void *v, *xn;
  float *rstd_post, *rstd_pre;
};
struct NormBwd {
  int T, d, k;
  const void *dv, *dxn, *v, *y, *y_perm, *y_add, *w_post, *w_pre;
  const float *gates, *gate, *rstd_post, *rstd_pre;
  const int32_t* slot_row;
  float res_scale;
  void *dx, *dy, *dy_perm;
  float *dgates, *dgate, *dw_post, *dw_pre;
  float* part;  // workspace: norm_workspace_bytes
};
size_t norm_workspace_bytes(int T, int d);
// elem_bytes: 2 (bf16) or 4 (float)
hipError_t block_norm_forward(int elem_bytes, const NormFwd& a, hipStream_t st);
hipError_t block_norm_backward(int elem_bytes, const NormBwd& a, hipStream_t st);

}  // namespace moe
