// training_api.cu - C-ABI entry points of the operators around the expert
// layer in a training step (include/moe.h): argument checks, then the
// launches of score_route.cu, norm.cu, rms.cu, checkpoint.cu (decoding), xent.cu
// and clip.cu on the caller's stream.
#include <climits>
#include <cmath>

#include "internal.h"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }
bool aligned_or_null(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool type_ok(int t) { return t == MOE_TYPE_F32 || t == MOE_TYPE_BF16; }
size_t type_bytes(int t) { return t == MOE_TYPE_BF16 ? 2 : 4; }

// Arrays of T*top_k entries may be NULL when T == 0.
bool route_out_ok(const moe_route_out* r, int T) {
  if (!r) return false;
  const bool tok = T == 0 || (aligned(r->topk_idx, 16) && aligned(r->gate, 16) && aligned(r->row_of_assign, 16));
  return tok && aligned(r->counts, 16) && aligned(r->offsets, 16) && aligned(r->padded_offsets, 16) &&
         aligned(r->assign_of_row, 16);
}

bool norm_ok(const moe_norm_dims* d) {
  return d && d->T >= 0 && d->H >= 1 && d->H <= INT_MAX / 2 && d->ld_x >= d->H && d->ld_y >= d->H &&
         d->ld_dx >= d->H && type_ok(d->x_type) && type_ok(d->w_type) && std::isfinite(d->eps) &&
         d->eps >= 0.f;
}
NormDesc norm_desc(const moe_norm_dims* d) {
  return NormDesc{d->T, d->H, d->ld_x, d->ld_y, d->ld_dx, d->x_type, d->w_type, d->eps};
}

bool router_ok(const moe_router_dims* d) {
  if (!d || d->T < 0 || d->E < 1 || d->E > kMaxE || d->top_k < 1 || d->top_k > kMaxTopK || d->ld < d->E) return false;
  if (!type_ok(d->type) || (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID)) return false;
  if (d->groups < 1 || d->groups > 32 || d->E % d->groups || d->top_groups < 1 || d->top_groups > d->groups) return false;
  const int size = d->E / d->groups;
  if (d->group_top < 1 || d->group_top > 2 || d->group_top > size || d->top_k > d->top_groups * size) return false;
  if (!(d->scale >= 0x1p-64f && d->scale <= 0x1p64f)) return false;
  return (int64_t)d->T * d->top_k + (int64_t)kAlign * d->E < ((int64_t)1 << 31);
}

bool rms_ok(const moe_rms_dims* d) {
  return d && d->T >= 0 && d->H >= 1 && d->H <= INT_MAX / 2 && d->ld_x >= d->H && d->ld_residual >= d->H &&
         d->ld_h >= d->H && d->ld_y >= d->H && d->ld_dh >= d->H && d->ld_dx >= d->H && type_ok(d->x_type) &&
         type_ok(d->w_type) && std::isfinite(d->eps) && d->eps >= 0.f;
}

// Host checks of the cross entropy's dims: tile counts and coordinates stay
// in 31 bits.
moe_status xent_check(const moe_xent_dims* d) {
  if (!d || d->T < 0 || d->V < 1 || d->H < 1 || d->ld_x < d->H || d->ld_w < d->H)
    return MOE_ERR_INVALID_ARG;
  if (d->index_type != MOE_INDEX_I32 && d->index_type != MOE_INDEX_I64) return MOE_ERR_INVALID_ARG;
  if (d->H % 8 || d->ld_x % 8 || d->ld_w % 8) return MOE_ERR_UNSUPPORTED;
  if (d->T > (1 << 30) || d->V > (1 << 30) || d->H > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  auto tiles = [](int64_t n) { return (n + 255) / 256; };
  const int64_t t = tiles(d->T), h = tiles(d->H), v = tiles(d->V);
  // (192-column tiles and slices of K at most double a count)
  return t * v < (1 << 28) && t * h < (1 << 28) && v * h < (1 << 28) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}
XentDesc xent_desc(const moe_xent_dims* d) {
  return XentDesc{d->T, d->H, d->V, d->ld_x, d->ld_w, d->ignore_index, d->index_type, wait_limit_ns()};
}

bool grads_ok(const moe_grad_tensor* t, int count, bool clip) {
  if (count < 0 || (count > 0 && !t)) return false;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > ((int64_t)1 << 46) || !type_ok(t[i].type)) return false;
    total += t[i].n;
    if (total > ((int64_t)1 << 46)) return false;
    const size_t a = type_bytes(t[i].type);
    if (t[i].n > 0 && (!aligned(t[i].src, a) || (clip && !aligned(t[i].dst, a)))) return false;
  }
  return true;
}

moe_status grads(const moe_grad_tensor* t, int count, bool clip, float max_norm, float* norm, void* ws,
                 size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (!grads_ok(t, count, clip) || !aligned(norm, 4) || !aligned(dev_status, 16) || !aligned(ws, 16) ||
      ws_bytes < grad_workspace_bytes(count))
    return MOE_ERR_INVALID_ARG;
  if (clip && !(std::isfinite(max_norm) && max_norm >= 0.f)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_grad_clip(t, count, clip, max_norm, ws, norm,
                                      dev_status, static_cast<cudaStream_t>(stream)));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layer_norm(const moe_norm_dims* d, const void* x, const void* gamma, const void* beta,
                          void* y, float* mean, float* rstd, void* stream) {
  if (!norm_ok(d)) return MOE_ERR_INVALID_ARG;
  const size_t xa = type_bytes(d->x_type), wa = type_bytes(d->w_type);
  if (!aligned_or_null(gamma, wa) || !aligned_or_null(beta, wa) || !aligned_or_null(mean, 4) ||
      !aligned_or_null(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (d->T == 0) return MOE_OK;
  if (!aligned(x, xa) || !aligned(y, xa)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_layer_norm(norm_desc(d), x, gamma, beta, y, mean, rstd,
                                       static_cast<cudaStream_t>(stream)));
}

size_t moe_layer_norm_workspace_size(const moe_norm_dims* d) {
  if (!norm_ok(d)) return 0;
  const size_t n = (size_t)norm_partial_blocks(d->T) * 2 * d->H * sizeof(float);
  return n ? n : 16;
}

moe_status moe_layer_norm_backward(const moe_norm_dims* d, const void* dy, const void* x,
                                   const void* gamma, const float* mean, const float* rstd, void* dx,
                                   void* dgamma, void* dbeta, void* ws, size_t ws_bytes,
                                   void* stream) {
  if (!norm_ok(d)) return MOE_ERR_INVALID_ARG;
  const size_t xa = type_bytes(d->x_type), wa = type_bytes(d->w_type);
  if (!aligned_or_null(gamma, wa) || !aligned_or_null(dgamma, wa) || !aligned_or_null(dbeta, wa))
    return MOE_ERR_INVALID_ARG;
  if ((dgamma || dbeta) && (!aligned(ws, 16) || ws_bytes < moe_layer_norm_workspace_size(d)))
    return MOE_ERR_INVALID_ARG;
  if (d->T > 0 && (!aligned(dy, xa) || !aligned(x, xa) || !aligned(dx, xa) || !aligned(mean, 4) ||
                   !aligned(rstd, 4)))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_layer_norm_backward(norm_desc(d), dy, x, gamma, mean, rstd, dx, dgamma,
                                                dbeta, static_cast<float*>(ws),
                                                static_cast<cudaStream_t>(stream)));
}

size_t moe_router_workspace_size(const moe_router_dims* d) { return router_ok(d) ? router_workspace_bytes(*d) : 0; }

moe_status moe_router(const moe_router_dims* d, const void* logits, const float* bias, const moe_route_out* o,
                      void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (!router_ok(d) || !route_out_ok(o, d->T) || !aligned(ws, 16) || !aligned(dev_status, 16) ||
      ws_bytes < router_workspace_bytes(*d) || !aligned_or_null(bias, 4))
    return MOE_ERR_INVALID_ARG;
  if (d->T > 0 && !aligned(logits, type_bytes(d->type))) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_router(*d, logits, bias, *o, static_cast<uint16_t*>(ws), dev_status,
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_router_backward(const moe_router_dims* d, const moe_route_out* r, const void* logits,
                               const float* dgate, void* dlogits, int32_t* dev_status, void* stream) {
  if (!router_ok(d) || !r || !aligned(dev_status, 16)) return MOE_ERR_INVALID_ARG;
  if (d->T == 0) return MOE_OK;
  const size_t a = type_bytes(d->type);
  if (!aligned(r->topk_idx, 16) || !aligned(r->gate, 16) || !aligned(logits, a) || !aligned(dgate, 4) ||
      !aligned(dlogits, a))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_router_backward(*d, *r, logits, dgate, dlogits, dev_status,
                                            static_cast<cudaStream_t>(stream)));
}

moe_status moe_balance_bias(int E, const int32_t* counts, float rate, const float* bias, float* out, void* stream) {
  if (E < 1 || E > kMaxE || !std::isfinite(rate) || !aligned(counts, 4) || !aligned(bias, 4) || !aligned(out, 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_balance_bias(counts, E, rate, bias, out, static_cast<cudaStream_t>(stream)));
}

moe_status moe_rms_norm(const moe_rms_dims* d, const void* x, const void* residual, const void* gamma, void* h,
                        void* y, uint8_t* q, uint8_t* scales, float* rstd, void* stream) {
  if (!rms_ok(d)) return MOE_ERR_INVALID_ARG;
  const size_t xa = type_bytes(d->x_type), wa = type_bytes(d->w_type);
  if (!aligned_or_null(gamma, wa) || !aligned_or_null(rstd, 4) || !aligned_or_null(residual, xa) ||
      !aligned_or_null(h, xa) || !aligned_or_null(y, xa) || (h && !residual) || (h && h == y))
    return MOE_ERR_INVALID_ARG;
  if ((q || scales) && (d->H % 32 || !aligned(q, 16) || !scales)) return MOE_ERR_INVALID_ARG;
  if (d->T == 0) return MOE_OK;
  if (!aligned(x, xa)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_rms_norm(*d, x, residual, gamma, h, y, q, scales, rstd,
                                     static_cast<cudaStream_t>(stream)));
}

size_t moe_rms_norm_workspace_size(const moe_rms_dims* d) {
  if (!rms_ok(d)) return 0;
  const size_t n = (size_t)norm_partial_blocks(d->T) * d->H * sizeof(float);
  return n ? n : 16;
}

moe_status moe_rms_norm_backward(const moe_rms_dims* d, const void* dy, const void* h, const void* dh,
                                 const void* gamma, const float* rstd, void* dx, void* dgamma, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (!rms_ok(d)) return MOE_ERR_INVALID_ARG;
  const size_t xa = type_bytes(d->x_type), wa = type_bytes(d->w_type);
  if (!aligned_or_null(gamma, wa) || !aligned_or_null(dgamma, wa) || !aligned_or_null(dh, xa))
    return MOE_ERR_INVALID_ARG;
  if (dgamma && (!aligned(ws, 16) || ws_bytes < moe_rms_norm_workspace_size(d))) return MOE_ERR_INVALID_ARG;
  if (d->T > 0 && (!aligned(dy, xa) || !aligned(h, xa) || !aligned(dx, xa) || !aligned(rstd, 4)))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_rms_norm_backward(*d, dy, h, dh, gamma, rstd, dx, dgamma, static_cast<float*>(ws),
                                              static_cast<cudaStream_t>(stream)));
}

moe_status moe_dequantize_mxfp8(const uint8_t* q, const uint8_t* scales, int R, int C, int64_t ld, moe_type type,
                                void* dst, void* stream) {
  if (R < 0 || C < 0 || C % 32 || ld < C || !type_ok(type)) return MOE_ERR_INVALID_ARG;
  if ((int64_t)R * C == 0) return MOE_OK;
  if (!aligned(q, 16) || !scales || !aligned(dst, type_bytes(type))) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_dequantize(q, scales, R, C, ld, type, dst, static_cast<cudaStream_t>(stream)));
}

size_t moe_cross_entropy_workspace_size(const moe_xent_dims* d, int which) {
  if (xent_check(d) != MOE_OK) return 0;
  if (which == MOE_WS_FORWARD) return xent_forward_bytes(xent_desc(d));
  if (which == MOE_WS_BACKWARD) return xent_backward_bytes(xent_desc(d));
  return 0;
}

moe_status moe_cross_entropy(const moe_xent_dims* d, const void* X, const void* W, const void* targets,
                             float* loss, float* lse, float* total, void* ws, size_t ws_bytes,
                             int32_t* dev_status, void* stream) {
  const moe_status c = xent_check(d);
  if (c != MOE_OK) return c;
  if (!aligned(total, 4) || !aligned(dev_status, 16) || !aligned(ws, 16) ||
      ws_bytes < xent_forward_bytes(xent_desc(d)))
    return MOE_ERR_INVALID_ARG;
  const size_t ta = d->index_type == MOE_INDEX_I64 ? 8 : 4;
  if (d->T > 0 && (!aligned(X, 16) || !aligned(W, 16) || !aligned(targets, ta) || !aligned(loss, 4) ||
                   !aligned(lse, 4)))
    return MOE_ERR_INVALID_ARG;
  moe_status st;
  const cudaError_t e = launch_xent_forward(xent_desc(d), X, W, targets, loss, lse, total,
                                            static_cast<char*>(ws), dev_status,
                                            static_cast<cudaStream_t>(stream), &st);
  return e != cudaSuccess ? MOE_ERR_CUDA : st;
}

moe_status moe_cross_entropy_backward(const moe_xent_dims* d, const void* X, const void* W,
                                      const void* targets, const float* lse, const float* total,
                                      const float* dloss, moe_reduction reduction, void* dX, void* dW,
                                      void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const moe_status c = xent_check(d);
  if (c != MOE_OK) return c;
  if (reduction < MOE_REDUCE_NONE || reduction > MOE_REDUCE_MEAN) return MOE_ERR_INVALID_ARG;
  if (!aligned(dev_status, 16) || !aligned(ws, 16) || ws_bytes < xent_backward_bytes(xent_desc(d)) ||
      !aligned_or_null(dX, 16) || !aligned_or_null(dW, 16))
    return MOE_ERR_INVALID_ARG;
  const size_t ta = d->index_type == MOE_INDEX_I64 ? 8 : 4;
  if (d->T > 0 && (!aligned(X, 16) || !aligned(W, 16) || !aligned(targets, ta) || !aligned(lse, 4) ||
                   !aligned(dloss, 4) || (reduction == MOE_REDUCE_MEAN && !aligned(total, 4))))
    return MOE_ERR_INVALID_ARG;
  moe_status st;
  const cudaError_t e = launch_xent_backward(xent_desc(d), X, W, targets, lse, total, dloss, reduction,
                                             dX, dW, static_cast<char*>(ws), dev_status,
                                             static_cast<cudaStream_t>(stream), &st);
  return e != cudaSuccess ? MOE_ERR_CUDA : st;
}

size_t moe_grad_workspace_size(int count) { return count < 0 ? 0 : grad_workspace_bytes(count); }

moe_status moe_grad_norm(const moe_grad_tensor* t, int count, float* norm, void* ws, size_t ws_bytes,
                         int32_t* dev_status, void* stream) {
  return grads(t, count, false, 0.f, norm, ws, ws_bytes, dev_status, stream);
}

moe_status moe_clip_grads(const moe_grad_tensor* t, int count, float max_norm, float* norm, void* ws,
                          size_t ws_bytes, int32_t* dev_status, void* stream) {
  return grads(t, count, true, max_norm, norm, ws, ws_bytes, dev_status, stream);
}

}  // extern "C"
