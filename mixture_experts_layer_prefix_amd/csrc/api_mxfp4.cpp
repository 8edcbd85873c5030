// C ABI of the weights in 4 bits and of the routed experts of a few tokens on
// them.  Arguments are validated here before any launch; see include/moe.h.
#include "checks.h"
#include "mxfp4.h"

using namespace moe;

namespace {

// A launch over a matrix takes 16 threads a row in x and a workgroup for every
// 512 columns in y: threads in x stay below 2^32, workgroups in y below 2^16.
constexpr int64_t kMaxRows = (1 << 28) - 16, kMaxCols = 1 << 24;

moe_status check_matrix(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols % 128) return MOE_EINVAL;
  return rows > kMaxRows || cols > kMaxCols ? MOE_EUNSUPPORTED : MOE_OK;
}

// I_shared and n_shared are not read.  Byte offsets inside the tokens, h, an
// expert's codes and all experts' scales fit in 31 or 32 bits.
moe_status check_ffn(const moe_dims* D) {
  if (!D || D->T < 0 || D->d < 1 || D->I < 1 || D->E < 1 || D->E > 1024 || D->k < 1 || D->k > 16) return MOE_EINVAL;
  if (D->T > kMaxTokens || D->d % 128 || D->I % 128 || (int64_t)D->I * D->d > UINT32_MAX ||
      D->T * D->d > INT32_MAX || D->T * D->k > INT32_MAX / D->I ||
      (int64_t)D->E * D->I > (int64_t)32 * UINT32_MAX / D->d)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

}  // namespace

namespace moe {

moe_status routed_ffn_workspace_bytes(const moe_dims* dims, size_t* bytes) {
  MOE_TRY(check_ffn(dims));
  *bytes = routed_ffn_scratch_bytes(dims->T, dims->d, dims->E, dims->k, dims->I);
  return MOE_OK;
}

}  // namespace moe

extern "C" {

moe_status moe_quantize_mxfp4(const void* src_bf16, int64_t rows, int64_t cols, uint8_t* dst, uint8_t* scale,
                              void* stream) {
  MOE_TRY(check_matrix(rows, cols));
  if (rows == 0 || cols == 0) return MOE_OK;  // empty tensors may have no address
  if (!need(src_bf16, 16) || !need(dst, 16) || !need(scale, 4)) return MOE_EINVAL;
  return done(launch_quantize_mxfp4(static_cast<const bf16_t*>(src_bf16), rows, cols, dst, scale,
                                    static_cast<hipStream_t>(stream)));
}

moe_status moe_dequantize_mxfp4(const uint8_t* src, const uint8_t* scale, int64_t rows, int64_t cols, void* dst_bf16,
                                void* stream) {
  MOE_TRY(check_matrix(rows, cols));
  if (rows == 0 || cols == 0) return MOE_OK;
  if (!need(src, 16) || !need(scale, 4) || !need(dst_bf16, 16)) return MOE_EINVAL;
  return done(launch_dequantize_mxfp4(src, scale, rows, cols, static_cast<bf16_t*>(dst_bf16),
                                      static_cast<hipStream_t>(stream)));
}

moe_status moe_routed_ffn_mxfp4(const moe_dims* dims, const uint8_t* x, const uint8_t* x_scale,
                                const int32_t* topk_idx, const float* topk_w, const moe_weights_mxfp4* w,
                                const void* y_add, void* y, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_ffn(dims));
  if (dims->T == 0) return MOE_OK;  // empty tensors may have no address
  if (!need(x, 16) || !need(x_scale, 4) || !need(topk_idx, 4) || !need(topk_w, 4) || !w || !aligned_to(y_add, 16) ||
      !need(y, 16))
    return MOE_EINVAL;
  for (const uint8_t* q : {w->q_gate, w->q_up, w->q_down})
    if (!need(q, 16)) return MOE_EINVAL;
  for (const uint8_t* q : {w->q_gate_scale, w->q_up_scale, w->q_down_scale})
    if (!need(q, 4)) return MOE_EINVAL;
  MOE_TRY(check_scratch(ws, ws_bytes, routed_ffn_scratch_bytes(dims->T, dims->d, dims->E, dims->k, dims->I)));
  RoutedFfn p = {};
  p.T = dims->T;
  p.d = dims->d;
  p.E = dims->E;
  p.k = dims->k;
  p.I = dims->I;
  p.x = x;
  p.x_scale = x_scale;
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  p.w = *w;
  p.y_add = static_cast<const bf16_t*>(y_add);
  p.y = static_cast<bf16_t*>(y);
  return done(launch_routed_ffn(p, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
