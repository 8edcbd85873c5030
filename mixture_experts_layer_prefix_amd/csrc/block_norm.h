// Arguments of the block norm kernels (see block_norm.hip).
#pragma once
#include "common.h"

namespace moe {

struct BlockNorm {
  int64_t T, gate_every;
  int d, post_norm;
  float alpha, beta, eps;
  const void *x, *y;                    // residual; block output or null
  const float *w_post, *gate, *w_pre;   // each or null
  void *x_out, *a;                      // a null: no norm of x' (or its codes alone)
  uint8_t *a_q, *a_scale;               // E4M3 codes and block scales of the bf16 a, or both null
  float *r_post, *r_pre;                // each or null
};

struct BlockNormBwd {
  int64_t T, gate_every, per, ldp;      // rows per team; row stride of the partial sums
  int d, post_norm;
  float alpha, beta;
  const void *dx_out, *da, *x_out, *y;  // gradients of x' and a, each or null; x'; block output or null
  const float *r_post, *r_pre, *w_post, *gate, *w_pre;
  void *dx, *dy;
  float *dw_post, *dgate, *dw_pre;      // each or null
  float *part_pre, *part_post, *part_gate;
};

size_t block_norm_scratch_bytes(int64_t T, int d);
hipError_t launch_block_norm(bool act_f32, bool res_f32, const BlockNorm& p, hipStream_t s);
hipError_t launch_block_norm_bwd(bool act_f32, bool res_f32, BlockNormBwd p, void* scratch, hipStream_t s);

}  // namespace moe
