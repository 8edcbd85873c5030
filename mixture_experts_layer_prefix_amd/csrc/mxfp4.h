// Weights of E2M1 codes with a scale per 32 (mxfp4.hip) and the routed experts
// of a few tokens on them (routed_ffn.hip).
#pragma once
#include "common.h"

namespace moe {

// rows x cols (a multiple of 128) bf16 <-> codes [rows][cols/2] and scales [cols/128][rows][4].
hipError_t launch_quantize_mxfp4(const bf16_t* src, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scale,
                                 hipStream_t s);
hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scale, int64_t rows, int64_t cols, bf16_t* dst,
                                   hipStream_t s);

struct RoutedFfn {
  int64_t T;
  int d, E, k, I;
  const uint8_t *x, *x_scale;    // tokens [T][d] E4M3, [T][d/32]
  const int32_t* topk_idx;       // [T][k]
  const float* topk_w;           // [T][k]
  moe_weights_mxfp4 w;
  const bf16_t* y_add;           // [T][d] or null
  bf16_t* y;                     // [T][d]
};

size_t routed_ffn_scratch_bytes(int64_t T, int d, int E, int k, int I);
hipError_t launch_routed_ffn(const RoutedFfn& p, void* scratch, hipStream_t s);

}  // namespace moe
