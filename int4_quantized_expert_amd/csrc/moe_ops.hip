// moe_ops.hip — the C entries of the operators beside the layer of include/moe.h: argument validation before
// anything is enqueued. Nothing here synchronizes, allocates device memory or keeps state.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

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

constexpr int kMaxAdapters = 1024, kMaxRank = 128, kMaxGrads = 65536;
constexpr int64_t kMaxGradElems = (int64_t)1 << 40;

// sizes only
int check_adapters(const moe_adapters* d) {
  if (!d) return MOE_OK;
  if (d->n_adapters < 1 || d->n_adapters > kMaxAdapters) return MOE_E_SHAPE;
  return d->rank >= 8 && d->rank <= kMaxRank && d->rank % 8 == 0 ? MOE_OK : MOE_E_SHAPE;
}
int check_adapter_arrays(const moe_adapters* d, const int32_t* ids) {
  if (!d) return MOE_OK;
  if (!d->a || !d->b || !d->scale) return MOE_E_NULL;
  return aligned16(d->a) && aligned16(d->b) && aligned(d->scale, 4) && aligned(ids, 4) ? MOE_OK : MOE_E_ARG;
}

int check_grads(const moe_grad* g, int32_t count) {
  if (!g) return MOE_E_NULL;
  if (count < 1 || count > kMaxGrads) return MOE_E_SHAPE;
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    if (g[i].n < 0 || g[i].n > kMaxGradElems) return MOE_E_SHAPE;
    if (!dtype_ok(g[i].dtype)) return MOE_E_ARG;
    if (g[i].n == 0) continue;
    if (!g[i].g || !g[i].out) return MOE_E_NULL;
    if (!elem_aligned(g[i].g, g[i].dtype) || !elem_aligned(g[i].out, g[i].dtype)) return MOE_E_ARG;
    chunks += clip_chunks(g + i, 1);
    if (chunks > (1 << 30)) return MOE_E_SHAPE;
  }
  return MOE_OK;
}

// Whether an out overlaps another tensor, or its own g in part.
bool grads_overlap(const moe_grad* g, int32_t count) {
  struct Span {
    uintptr_t a, b;
    int i;
  };
  std::vector<Span> outs;
  auto bytes = [&](int i) { return (uintptr_t)g[i].n * (g[i].dtype == MOE_DTYPE_F32 ? 4 : 2); };
  for (int i = 0; i < count; ++i)
    if (g[i].n > 0) {
      const uintptr_t o = reinterpret_cast<uintptr_t>(g[i].out);
      outs.push_back({o, o + bytes(i), i});
    }
  std::sort(outs.begin(), outs.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  for (size_t k = 1; k < outs.size(); ++k)
    if (outs[k].a < outs[k - 1].b) return true;
  for (int i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].g), b = a + bytes(i);
    // the outs are disjoint and in order: the first that ends behind a, and those that follow until b
    auto it = std::upper_bound(outs.begin(), outs.end(), a, [](uintptr_t v, const Span& s) { return v < s.b; });
    for (; it != outs.end() && it->a < b; ++it)
      if (it->i != i || it->a != a) return true;
  }
  return false;
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

size_t moe_linear_adapted_workspace_bytes(const moe_linear_config* cfg, const moe_adapters* adapters, int32_t max_tokens) {
  if (check_linear(cfg) != MOE_OK || check_adapters(adapters) != MOE_OK || !tokens_ok(max_tokens)) return 0;
  return adapted_ws_bytes(*cfg, adapters, max_tokens);
}

int32_t moe_linear_adapted(const moe_linear_config* cfg, const uint8_t* codes, const float* scales, const float* bias,
                           const moe_adapters* adapters, const int32_t* ids, const void* x, int64_t ldx, int32_t T,
                           int32_t dtype, const void* residual, int64_t ldr, void* y, int64_t ldy, void* pre, int64_t ldp,
                           void* ws, size_t ws_bytes, hipStream_t stream) {
  int rc = check_linear(cfg);
  if (rc || (rc = check_adapters(adapters))) return rc;
  if (!codes || !scales || !x || !y) return MOE_E_NULL;
  if (!tokens_ok(T)) return MOE_E_SHAPE;
  const int64_t out = cfg->act == MOE_ACT_SWIGLU ? cfg->rows / 2 : cfg->rows;
  if (!dtype_ok(dtype) || ldx < cfg->cols || ldy < out || (residual && ldr < out) || (pre && ldp < cfg->rows))
    return MOE_E_ARG;
  if (!aligned16(codes) || !aligned(scales, 4) || !aligned(bias, 4)) return MOE_E_ARG;
  if (!elem_aligned(x, dtype) || !elem_aligned(residual, dtype) || !elem_aligned(y, dtype) || !elem_aligned(pre, dtype))
    return MOE_E_ARG;
  if ((rc = check_adapter_arrays(adapters, ids))) return rc;
  if ((rc = check_space(ws, ws_bytes, adapted_ws_bytes(*cfg, adapters, T)))) return rc;
  return done(launch_linear_adapted(*cfg, codes, scales, bias, adapters, ids, x, ldx, T, dtype, residual, ldr, y, ldy, pre,
                                    ldp, ws, stream));
}

size_t moe_linear_backward_workspace_bytes(const moe_linear_config* cfg, const moe_adapters* adapters,
                                           int32_t max_tokens) {
  if (check_linear(cfg) != MOE_OK || check_adapters(adapters) != MOE_OK || !tokens_ok(max_tokens)) return 0;
  return linear_grad_ws_bytes(*cfg, adapters, max_tokens);
}

int32_t moe_linear_backward(const moe_linear_config* cfg, const uint8_t* codes, const float* scales,
                            const moe_adapters* adapters, const int32_t* ids, const void* x, int64_t ldx, int32_t T,
                            int32_t dtype, const void* pre, int64_t ldp, const void* dy, int64_t ldd,
                            const void* residual, int64_t ldr, void* dx, int64_t ldg, void* d_a, void* d_b, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  int rc = check_linear(cfg);
  if (rc || (rc = check_adapters(adapters))) return rc;
  const bool act = cfg->act != MOE_ACT_NONE, ab = d_a || d_b;
  if (!codes || !scales || !dy || (act && !pre) || (!dx && !ab)) return MOE_E_NULL;
  if ((ab && (!adapters || !x)) || (residual && !dx)) return MOE_E_NULL;
  if (!tokens_ok(T)) return MOE_E_SHAPE;
  const int64_t out = cfg->act == MOE_ACT_SWIGLU ? cfg->rows / 2 : cfg->rows;
  if (!dtype_ok(dtype) || ldd < out || (act && ldp < cfg->rows) || (ab && ldx < cfg->cols) || (dx && ldg < cfg->cols) ||
      (residual && ldr < cfg->cols))
    return MOE_E_ARG;
  if (!aligned16(codes) || !aligned(scales, 4) || !aligned16(d_a) || !aligned16(d_b)) return MOE_E_ARG;
  for (const void* p : {x, pre, dy, residual, (const void*)dx})
    if (!elem_aligned(p, dtype)) return MOE_E_ARG;
  if ((rc = check_adapter_arrays(adapters, ids))) return rc;
  if ((rc = check_space(ws, ws_bytes, linear_grad_ws_bytes(*cfg, adapters, T)))) return rc;
  return done(launch_linear_grad(*cfg, codes, scales, adapters, ids, x, ldx, T, dtype, pre, ldp, dy, ldd, residual, ldr, dx,
                                 ldg, d_a, d_b, ws, stream));
}

size_t moe_grad_table_bytes(const moe_grad* grads, int32_t count) {
  return check_grads(grads, count) == MOE_OK ? clip_table_bytes(grads, count) : 0;
}

int32_t moe_grad_table(const moe_grad* grads, int32_t count, void* table, size_t table_bytes, moe_grads* out,
                       hipStream_t stream) {
  const int rc = check_grads(grads, count);
  if (rc) return rc;
  if (!out) return MOE_E_NULL;
  try {
    if (grads_overlap(grads, count)) return MOE_E_ARG;
  } catch (const std::bad_alloc&) {
    return MOE_E_NOMEM;
  }
  if (check_space(table, table_bytes, clip_table_bytes(grads, count))) return MOE_E_WORKSPACE;
  *out = moe_grads{count, clip_chunks(grads, count), table};
  return done(launch_clip_table(grads, count, table, stream));
}

int32_t moe_grad_clip(const moe_grads* grads, float max_norm, float* norm, hipStream_t stream) {
  if (!grads || !norm) return MOE_E_NULL;
  if (grads->count < 1 || grads->count > kMaxGrads || grads->chunks < 0) return MOE_E_SHAPE;
  if (!grads->table || !aligned(grads->table, 256)) return MOE_E_WORKSPACE;
  if (!(max_norm > 0.0f) || !aligned(norm, 4)) return MOE_E_ARG;
  return done(launch_clip(*grads, max_norm, norm, stream));
}

}  // extern "C"
