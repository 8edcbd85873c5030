// C ABI of the operators around the layer: routed tokens sorted by expert and
// back, the norms before and after a residual block, gradient clipping.
// Arguments are validated here before any launch; see include/moe.h.
#include <math.h>

#include "block_norm.h"
#include "clip.h"

using namespace moe;

namespace {

// Workgroups times threads of a launch stay below 2^32.
constexpr int64_t kMaxTokens = 4194303;
constexpr int kMaxNormDim = 16384;
// The row kernels count columns in an int, in steps of at most 8,192.
constexpr int kMaxRowDim = 1 << 30;

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool need(const void* p, size_t n) { return p && aligned_to(p, n); }

size_t elem(moe_prec prec) { return prec == MOE_F32 ? 4 : 2; }

moe_status check_prec(moe_prec prec) {
  if (prec == MOE_MXFP8) return MOE_EUNSUPPORTED;
  return prec == MOE_F32 || prec == MOE_BF16 ? MOE_OK : MOE_EINVAL;
}

// E is read by the sort alone.
moe_status check_routes(const moe_dims* D, moe_prec prec, bool experts) {
  if (!D || D->T < 0 || D->d < 1 || D->k < 1 || D->k > 16) return MOE_EINVAL;
  if (experts && (D->E < 1 || D->E > 1024)) return MOE_EINVAL;
  if (D->T > kMaxTokens || D->d > kMaxRowDim) return MOE_EUNSUPPORTED;
  return check_prec(prec);
}

moe_status check_block(const moe_block* b, moe_prec prec, bool gate) {
  if (!b || b->T < 0 || b->d < 1 || (gate && b->gate_every < 1)) return MOE_EINVAL;
  if (!isfinite(b->alpha) || !isfinite(b->beta) || !isfinite(b->eps) || !(b->eps > 0.0f)) return MOE_EINVAL;
  if (b->T > kMaxTokens || b->d > kMaxNormDim) return MOE_EUNSUPPORTED;
  return check_prec(prec);
}

moe_status check_grads(const void* const* grads, const int64_t* numel, const int32_t* types, int32_t n) {
  if (n < 0 || (n > 0 && (!grads || !numel || !types))) return MOE_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] < 0) return MOE_EINVAL;
    if (types[i] != MOE_F32 && types[i] != MOE_BF16) return types[i] == MOE_MXFP8 ? MOE_EUNSUPPORTED : MOE_EINVAL;
    if (numel[i] > 0 && !need(grads[i], types[i] == MOE_F32 ? 4 : 2)) return MOE_EINVAL;
  }
  return MOE_OK;
}

moe_status check_scratch(const void* ws, size_t bytes, size_t required) {
  if (required && (!ws || bytes < required)) return MOE_EWORKSPACE;
  return aligned_to(ws, 16) ? MOE_OK : MOE_EINVAL;
}

moe_status done(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

#define MOE_TRY(expr)              \
  do {                             \
    moe_status st_ = (expr);       \
    if (st_ != MOE_OK) return st_; \
  } while (0)

}  // namespace

namespace moe {

// moe_workspace_bytes, which = 5.
moe_status sort_workspace_bytes(const moe_dims* dims, moe_prec prec, size_t* bytes) {
  MOE_TRY(check_routes(dims, prec, true));
  *bytes = sort_scratch_bytes(dims->T, dims->k, dims->E);
  return MOE_OK;
}

}  // namespace moe

extern "C" {

moe_status moe_sort_tokens(const moe_dims* dims, moe_prec prec, const int32_t* topk_idx, const void* x,
                           int32_t* expert_counts, int32_t* expert_offsets, int32_t* row_token, int32_t* token_row,
                           void* x_perm, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_routes(dims, prec, true));
  if (!need(expert_counts, 4) || !need(expert_offsets, 4)) return MOE_EINVAL;
  if (dims->T > 0) {
    if (!need(topk_idx, 4) || !need(row_token, 4) || !need(token_row, 4)) return MOE_EINVAL;
    if (x_perm && (!need(x, elem(prec)) || !need(x_perm, elem(prec)) || x == x_perm)) return MOE_EINVAL;
  }
  MOE_TRY(check_scratch(ws, ws_bytes, sort_scratch_bytes(dims->T, dims->k, dims->E)));
  return done(launch_sort(prec == MOE_F32, topk_idx, x, dims->T, dims->d, dims->E, dims->k, expert_counts,
                          expert_offsets, row_token, token_row, x_perm, ws, static_cast<hipStream_t>(stream)));
}

moe_status moe_sort_tokens_backward(const moe_dims* dims, moe_prec prec, const void* dx_perm, const int32_t* token_row,
                                    const void* dx_add, void* dx, void* stream) {
  MOE_TRY(check_routes(dims, prec, false));
  if (dims->T == 0) return MOE_OK;
  const size_t n = elem(prec);
  if (!need(dx_perm, n) || !need(token_row, 4) || !aligned_to(dx_add, n) || !need(dx, n) || dx == dx_perm)
    return MOE_EINVAL;
  return done(launch_unsort(prec == MOE_F32, dx_perm, token_row, nullptr, dx_add, dx, dims->T, dims->d, dims->k,
                            static_cast<hipStream_t>(stream)));
}

moe_status moe_unsort_tokens(const moe_dims* dims, moe_prec prec, const void* o_perm, const int32_t* token_row,
                             const float* topk_w, const void* y_add, void* y, void* stream) {
  MOE_TRY(check_routes(dims, prec, false));
  if (dims->T == 0) return MOE_OK;
  const size_t n = elem(prec);
  if (!need(o_perm, n) || !need(token_row, 4) || !need(topk_w, 4) || !aligned_to(y_add, n) || !need(y, n) ||
      y == o_perm)
    return MOE_EINVAL;
  return done(launch_unsort(prec == MOE_F32, o_perm, token_row, topk_w, y_add, y, dims->T, dims->d, dims->k,
                            static_cast<hipStream_t>(stream)));
}

moe_status moe_unsort_tokens_backward(const moe_dims* dims, moe_prec prec, const void* dy, const void* o_perm,
                                      const int32_t* token_row, const float* topk_w, void* do_perm, float* dtopk_w,
                                      void* stream) {
  MOE_TRY(check_routes(dims, prec, false));
  if (dims->T == 0) return MOE_OK;  // empty tensors may have no address
  if (!do_perm && !dtopk_w) return MOE_EINVAL;
  const size_t n = elem(prec);
  if (!need(dy, n) || !need(token_row, 4)) return MOE_EINVAL;
  if (do_perm && (!aligned_to(do_perm, n) || !need(topk_w, 4) || do_perm == o_perm || do_perm == dy))
    return MOE_EINVAL;
  if (dtopk_w && (!aligned_to(dtopk_w, 4) || !need(o_perm, n) || dtopk_w == topk_w)) return MOE_EINVAL;
  return done(launch_unsort_bwd(prec == MOE_F32, dy, o_perm, token_row, topk_w, do_perm, dtopk_w, dims->T, dims->d,
                                dims->k, static_cast<hipStream_t>(stream)));
}

moe_status moe_block_norm(const moe_block* block, moe_prec prec, const void* x, const void* y, const float* w_post,
                          const float* gate, const float* w_pre, void* x_out, void* a, float* r_post, float* r_pre,
                          void* stream) {
  MOE_TRY(check_block(block, prec, gate != nullptr));
  if (block->T == 0) return MOE_OK;  // empty tensors may have no address
  if (!y && (!a || x_out || gate || block->post_norm)) return MOE_EINVAL;
  if ((w_post || r_post) && !block->post_norm) return MOE_EINVAL;
  if ((w_pre || r_pre) && !a) return MOE_EINVAL;
  const size_t na = elem(prec), nr = block->res_f32 ? 4 : na;
  if (!need(x, nr) || !aligned_to(y, na) || (y && !need(x_out, nr)) || !aligned_to(a, na)) return MOE_EINVAL;
  for (const void* p : {(const void*)w_post, (const void*)gate, (const void*)w_pre, (const void*)r_post,
                        (const void*)r_pre})
    if (!aligned_to(p, 4)) return MOE_EINVAL;
  BlockNorm p = {};
  p.T = block->T;
  p.gate_every = block->gate_every;
  p.d = block->d;
  p.post_norm = block->post_norm != 0;
  p.alpha = block->alpha;
  p.beta = block->beta;
  p.eps = block->eps;
  p.x = x;
  p.y = y;
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.x_out = x_out;
  p.a = a;
  p.r_post = r_post;
  p.r_pre = r_pre;
  return done(launch_block_norm(prec == MOE_F32, prec == MOE_F32 || block->res_f32, p,
                                static_cast<hipStream_t>(stream)));
}

size_t moe_block_norm_scratch_bytes(int64_t T, int32_t d) {
  return T < 0 || d < 1 || T > kMaxTokens || d > kMaxNormDim ? 0 : block_norm_scratch_bytes(T, d);
}

moe_status moe_block_norm_backward(const moe_block* block, moe_prec prec, const void* dx_out, const void* da,
                                   const void* x_out, const void* y, const float* r_post, const float* r_pre,
                                   const float* w_post, const float* gate, const float* w_pre, void* dx, void* dy,
                                   float* dw_post, float* dgate, float* dw_pre, void* ws, size_t ws_bytes,
                                   void* stream) {
  MOE_TRY(check_block(block, prec, gate != nullptr));
  if (block->T > 0) {  // empty tensors may have no address
    if (!dx_out && !da) return MOE_EINVAL;
    if ((y != nullptr) != (dy != nullptr) || (!y && (gate || block->post_norm))) return MOE_EINVAL;
    if ((w_post || r_post) && !block->post_norm) return MOE_EINVAL;
    if ((w_pre || r_pre) && !da) return MOE_EINVAL;
  }
  if ((dw_post && !w_post) || (dgate && !gate) || (dw_pre && !w_pre)) return MOE_EINVAL;
  const size_t na = elem(prec), nr = block->res_f32 ? 4 : na;
  for (const void* p : {(const void*)w_post, (const void*)gate, (const void*)w_pre, (const void*)r_post,
                        (const void*)r_pre, (const void*)dw_post, (const void*)dgate, (const void*)dw_pre})
    if (!aligned_to(p, 4)) return MOE_EINVAL;
  if (block->T > 0) {
    if (!aligned_to(dx_out, nr) || !aligned_to(da, na) || !need(dx, nr) || !aligned_to(y, na) || !aligned_to(dy, na))
      return MOE_EINVAL;
    if (da && (!need(x_out, nr) || !r_pre)) return MOE_EINVAL;
    if (block->post_norm && !r_post) return MOE_EINVAL;
  }
  MOE_TRY(check_scratch(ws, ws_bytes, block_norm_scratch_bytes(block->T, block->d)));
  BlockNormBwd p = {};
  p.T = block->T;
  p.gate_every = block->gate_every;
  p.d = block->d;
  p.post_norm = block->post_norm != 0;
  p.alpha = block->alpha;
  p.beta = block->beta;
  p.dx_out = dx_out;
  p.da = da;
  p.x_out = x_out;
  p.y = y;
  p.r_post = r_post;
  p.r_pre = r_pre;
  p.w_post = w_post;
  p.gate = gate;
  p.w_pre = w_pre;
  p.dx = dx;
  p.dy = dy;
  p.dw_post = dw_post;
  p.dgate = dgate;
  p.dw_pre = dw_pre;
  return done(launch_block_norm_bwd(prec == MOE_F32, prec == MOE_F32 || block->res_f32, p, ws,
                                    static_cast<hipStream_t>(stream)));
}

size_t moe_grad_norm_scratch_bytes(const int64_t* numel, int32_t n) {
  if (n < 0 || (n > 0 && !numel)) return 0;
  return grad_norm_scratch_bytes(n, numel);
}

moe_status moe_grad_norm(const void* const* grads, const int64_t* numel, const int32_t* types, int32_t n, float* norm,
                         void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_grads(grads, numel, types, n));
  if (!need(norm, 4)) return MOE_EINVAL;
  MOE_TRY(check_scratch(ws, ws_bytes, grad_norm_scratch_bytes(n, numel)));
  return done(launch_grad_norm(n, grads, numel, types, norm, ws, static_cast<hipStream_t>(stream)));
}

moe_status moe_clip_grads(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* types,
                          int32_t n, float max_norm, const float* norm_in, float* norm, void* ws, size_t ws_bytes,
                          void* stream) {
  MOE_TRY(check_grads(grads, numel, types, n));
  MOE_TRY(check_grads(out, numel, types, n));
  if (!isfinite(max_norm) || max_norm < 0.0f || !aligned_to(norm_in, 4)) return MOE_EINVAL;
  if (!norm_in) {
    if (!need(norm, 4)) return MOE_EINVAL;
    MOE_TRY(check_scratch(ws, ws_bytes, grad_norm_scratch_bytes(n, numel)));
  }
  return done(launch_clip_grads(n, grads, out, numel, types, max_norm, norm_in, norm, ws,
                                static_cast<hipStream_t>(stream)));
}

}  // extern "C"
