// moe_ops.hip — the C entries of the routing and linear operators of include/moe.h: argument validation before
// anything is enqueued. Nothing here synchronizes, allocates or keeps state.
#include <cmath>

#include "moe_ops.h"

using namespace moe;

namespace {

constexpr int kMaxRows = 1 << 20, kMaxCols = 65536;
constexpr int32_t kMaxOpTokens = 1 << 20;

int check_route(const moe_route_config* c) {
  if (!c) return MOE_E_NULL;
  if (c->n_experts < 1 || c->n_experts > kMaxExperts) return MOE_E_SHAPE;
  if (c->n_group < 1 || c->n_group > kMaxGroups || c->n_experts % c->n_group != 0) return MOE_E_SHAPE;
  if (c->topk_group < 1 || c->topk_group > c->n_group) return MOE_E_SHAPE;
  if (c->top_k < 1 || c->top_k > kMaxTopK || c->top_k > c->topk_group * (c->n_experts / c->n_group)) return MOE_E_SHAPE;
  if (c->score != MOE_SCORE_SIGMOID && c->score != MOE_SCORE_SOFTMAX) return MOE_E_ARG;
  if (c->group_score != MOE_GROUP_TOP2 && c->group_score != MOE_GROUP_MAX) return MOE_E_ARG;
  if (c->renorm != 0 && c->renorm != 1) return MOE_E_ARG;
  if (!std::isfinite(c->scale) || c->scale <= 0.0f) return MOE_E_ARG;
  return MOE_OK;
}

bool dtype_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool elem_aligned(const void* p, int32_t dtype) { return aligned(p, dtype == MOE_DTYPE_F32 ? 4 : 2); }
bool tokens_ok(int32_t T) { return T >= 1 && T <= kMaxOpTokens; }

int check_space(const void* ws, size_t have, size_t need) {
  return ws && aligned(ws, 256) && have >= need ? MOE_OK : MOE_E_WORKSPACE;
}

int check_linear(const moe_linear_config* c) {
  if (!c) return MOE_E_NULL;
  if (c->rows <= 0 || c->rows % 64 != 0 || c->rows > kMaxRows) return MOE_E_SHAPE;
  if (c->cols <= 0 || c->cols % 32 != 0 || c->cols > kMaxCols) return MOE_E_SHAPE;
  if (c->weight_bits > 0 && c->weight_bits != 4 && c->weight_bits != 8) return MOE_E_ARG;
  if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_SWIGLU) return MOE_E_ARG;
  if (c->group_size > 0) {
    const int g = c->group_size;
    if (c->weight_bits == 8 || g % 32 != 0 || ((g / 32) & (g / 32 - 1)) != 0) return MOE_E_ARG;
    if (c->cols % g != 0) return MOE_E_SHAPE;
  }
  return MOE_OK;
}

int check_slot_grad(const float* e_out, const int32_t* ids, const float* dy, int32_t T, int32_t K, int32_t H,
                    const float* d_w) {
  if (!e_out || !ids || !dy || !d_w) return MOE_E_NULL;
  if (!tokens_ok(T) || K < 1 || K > kMaxTopK || H < 4 || H % 4 != 0 || H > kMaxHidden) return MOE_E_SHAPE;
  if (!aligned16(e_out) || !aligned16(dy) || !aligned(ids, 4) || !aligned(d_w, 4)) return MOE_E_ARG;
  return MOE_OK;
}

int32_t done(hipError_t e) { return e == hipSuccess ? MOE_OK : hip_fail(e); }

}  // namespace

extern "C" {

size_t moe_route_workspace_bytes(const moe_route_config* cfg, int32_t max_tokens) {
  if (check_route(cfg) != MOE_OK || !tokens_ok(max_tokens)) return 0;
  return route_ws_bytes(cfg->n_experts, max_tokens);
}

int32_t moe_route(const moe_route_config* cfg, const void* logits, int32_t dtype, int64_t ld, int32_t T,
                  const float* bias, const uint8_t* valid, int32_t* ids, float* w, int32_t* load, float* importance,
                  void* ws, size_t ws_bytes, hipStream_t stream) {
  int rc = check_route(cfg);
  if (rc) return rc;
  if (!logits || !ids || !w) return MOE_E_NULL;
  if (!tokens_ok(T)) return MOE_E_SHAPE;
  if (!dtype_ok(dtype) || ld < cfg->n_experts) return MOE_E_ARG;
  if (!elem_aligned(logits, dtype) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(w, 4) || !aligned(load, 4) ||
      !aligned(importance, 4))
    return MOE_E_ARG;
  if ((load || importance) && (rc = check_space(ws, ws_bytes, route_ws_bytes(cfg->n_experts, T)))) return rc;
  return done(launch_moe_route(*cfg, logits, dtype, ld, T, bias, valid, ids, w, load, importance, ws, stream));
}

int32_t moe_route_backward(const moe_route_config* cfg, const void* logits, int32_t dtype, int64_t ld, int32_t T,
                           const uint8_t* valid, const int32_t* ids, const float* d_w, const float* d_importance,
                           void* d_logits, int64_t ld_d, hipStream_t stream) {
  int rc = check_route(cfg);
  if (rc) return rc;
  if (!logits || !ids || !d_logits || (!d_w && !d_importance)) return MOE_E_NULL;
  if (!tokens_ok(T)) return MOE_E_SHAPE;
  if (!dtype_ok(dtype) || ld < cfg->n_experts || ld_d < cfg->n_experts) return MOE_E_ARG;
  if (!elem_aligned(logits, dtype) || !elem_aligned(d_logits, dtype) || !aligned(ids, 4) || !aligned(d_w, 4) ||
      !aligned(d_importance, 4))
    return MOE_E_ARG;
  return done(
      launch_moe_route_grad(*cfg, logits, dtype, ld, T, valid, ids, d_w, d_importance, d_logits, ld_d, stream));
}

int32_t moe_slot_weight_grad(const float* e_out, const int32_t* ids, const float* dy, int32_t T, int32_t K, int32_t H,
                             float* d_w, hipStream_t stream) {
  const int rc = check_slot_grad(e_out, ids, dy, T, K, H, d_w);
  return rc ? rc : done(launch_slot_grad(e_out, ids, dy, T, K, H, 1u << 31, d_w, stream));  // every id >= 0 counts
}

int32_t moe_slot_weight_grad_experts(const float* e_out, const int32_t* ids, const float* dy, int32_t T, int32_t K,
                                     int32_t H, int32_t n_experts, float* d_w, hipStream_t stream) {
  const int rc = check_slot_grad(e_out, ids, dy, T, K, H, d_w);
  if (rc) return rc;
  if (n_experts < 1 || n_experts > kMaxExperts) return MOE_E_SHAPE;
  return done(launch_slot_grad(e_out, ids, dy, T, K, H, (uint32_t)n_experts, d_w, stream));
}

size_t moe_linear_workspace_bytes(const moe_linear_config* cfg, int32_t max_tokens) {
  if (check_linear(cfg) != MOE_OK || !tokens_ok(max_tokens)) return 0;
  return linear_ws_bytes(*cfg, max_tokens);
}

int32_t moe_linear(const moe_linear_config* cfg, const uint8_t* codes, const float* scales, const float* bias,
                   const void* x, int64_t ldx, int32_t T, int32_t dtype, const void* residual, int64_t ldr, void* y,
                   int64_t ldy, void* ws, size_t ws_bytes, hipStream_t stream) {
  int rc = check_linear(cfg);
  if (rc) return rc;
  if (!codes || !scales || !x || !y) return MOE_E_NULL;
  if (!tokens_ok(T)) return MOE_E_SHAPE;
  const int64_t out = cfg->act == MOE_ACT_SWIGLU ? cfg->rows / 2 : cfg->rows;
  if (!dtype_ok(dtype) || ldx < cfg->cols || ldy < out || (residual && ldr < out)) return MOE_E_ARG;
  if (!aligned16(codes) || !aligned(scales, 4) || !aligned(bias, 4)) return MOE_E_ARG;
  if (!elem_aligned(x, dtype) || !elem_aligned(residual, dtype) || !elem_aligned(y, dtype)) return MOE_E_ARG;
  if ((rc = check_space(ws, ws_bytes, linear_ws_bytes(*cfg, T)))) return rc;
  return done(launch_linear(*cfg, codes, scales, bias, x, ldx, T, dtype, residual, ldr, y, ldy, ws, stream));
}

}  // extern "C"
