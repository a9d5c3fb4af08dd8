// moe_ops.h — launches and workspaces of the operators beside the layer (k_route.hip, k_linear*.hip, k_adapt.hip,
// k_clip.hip), which the C entries in moe_ops.hip call.
#pragma once
#include "moe_internal.h"

namespace moe {

// routing from logits and its gradients
size_t route_ws_bytes(int E, int T);
hipError_t launch_moe_route(const moe_route_config& c, const void* logits, int dtype, int64_t ld, int T,
                            const float* bias, const uint8_t* valid, int32_t* ids, float* w, int32_t* load, float* imp,
                            void* ws, hipStream_t st);
hipError_t launch_moe_route_grad(const moe_route_config& c, const void* logits, int dtype, int64_t ld, int T,
                                 const uint8_t* valid, const int32_t* ids, const float* dw, const float* dimp, void* dz,
                                 int64_t ld_d, hipStream_t st);
// slots whose id, taken as unsigned, is not below id_end are dropped
hipError_t launch_slot_grad(const float* eout, const int32_t* ids, const float* dy, int T, int K, int H, uint32_t id_end,
                            float* dw, hipStream_t st);
// product over weight codes with its epilogue
size_t linear_ws_bytes(const moe_linear_config& c, int64_t T);
hipError_t launch_linear(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                         const void* x, int64_t ldx, int T, int dtype, const void* res, int64_t ldr, void* y,
                         int64_t ldy, void* ws, hipStream_t st);

// the same with adapters by token (ad may be NULL) and the values in front of the activation
size_t adapted_ws_bytes(const moe_linear_config& c, int R, int64_t T);
hipError_t launch_linear_adapted(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                                 const moe_adapters* ad, const int32_t* ids, const void* x, int64_t ldx, int T, int dtype,
                                 const void* res, int64_t ldr, void* y, int64_t ldy, void* pre, int64_t ldp, void* ws,
                                 hipStream_t st);
// gradients of it
size_t linear_grad_ws_bytes(const moe_linear_config& c, const moe_adapters* ad, int64_t T);
hipError_t launch_linear_grad(const moe_linear_config& c, const uint8_t* codes, const float* scales,
                              const moe_adapters* ad, const int32_t* ids, const void* x, int64_t ldx, int T, int dtype,
                              const void* pre, int64_t ldp, const void* dy, int64_t ldd, const void* res, int64_t ldr,
                              void* dx, int64_t ldg, void* da, void* db, void* ws, hipStream_t st);

// ------------------------------------------------------------ adapters (k_adapt.hip)
// A run of positions (tokens in the order of their adapters) of one adapter, for the gradients' sums over tokens.
struct AdaptChunk {
  int32_t e, p0, p1;
  int32_t slot;  // of the partial sums; -1: the adapter's only chunk
};
constexpr int kAdaptSlots = 32;  // cnt > len gives at most 2 cnt / len chunks, and T / len is at most 16
inline int adapt_chunk_len(int64_t T) { return (int)((T + 4095) / 4096 * 256); }  // at most 16 chunks of T positions
inline int64_t adapt_max_chunks(int64_t T, int n) { return T / adapt_chunk_len(T) + (T < n ? T : n) + 1; }
// What the gradients need beside the order of the positions.
struct AdaptTable {
  int32_t* offsets;  // [n + 1] first position of each adapter, and of the tokens without one
  int32_t* slot0;    // [n] first partial sum of an adapter of several chunks
  int32_t* n_chunks;
  AdaptChunk* chunks;
};
hipError_t launch_adapt_order(const int32_t* ids, int T, int n_ad, int32_t* order, int32_t* pos_ad, hipStream_t st,
                              const AdaptTable* table = nullptr);
// h[p][r] = scale * sum over c of x[order[p]][c] a[ad[p]][r][c], 0 without an adapter; ht, where given, the same as [R][ldt]
struct AdaptDown {
  const void* x;
  int64_t ldx;
  int32_t vec_x, T, C, R, n_ad;
  const int32_t* order;
  const int32_t* ad;
  const void* a;
  const float* scale;
  float* h;
  float* ht;
  int32_t ldt;
};
hipError_t launch_adapt_down(const AdaptDown& a, int dtype, hipStream_t st);
// out[e] = sum over e's positions of v[p][r] m[p][c]: [n][R][C], or with `rows` [n][C][R]
struct AdaptOuter {
  const void* m;
  int64_t ldm;
  int32_t vec_m, T, C, R, n_ad, rows;
  const int32_t* order;  // rows of m, nullptr: m's rows are positions
  const float* v;
  const float* vt;
  int32_t ldt;
  AdaptTable table;
  float* part;  // [kAdaptSlots][R][C]
  void* out;
};
hipError_t launch_adapt_outer(const AdaptOuter& a, int dtype, hipStream_t st);
// out [n][Q][M] = in [n][M][Q] transposed, for the adapters that tokens have
hipError_t launch_adapt_transpose(const void* in, int n, int M, int Q, int elem, const int32_t* offsets, void* out,
                                  hipStream_t st);

// ------------------------------------------------------------ gradients' norm (k_clip.hip)
int64_t clip_chunks(const moe_grad* g, int count);
size_t clip_table_bytes(const moe_grad* g, int count);
hipError_t launch_clip_table(const moe_grad* g, int count, void* table, hipStream_t st);
hipError_t launch_clip(const moe_grads& t, float max_norm, float* norm, hipStream_t st);

}  // namespace moe
