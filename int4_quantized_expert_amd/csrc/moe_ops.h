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
size_t adapted_ws_bytes(const moe_linear_config& c, const moe_adapters* ad, int64_t T);
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
// A run of positions (tokens in the order of their adapters) of one adapter.
struct AdaptChunk {
  int32_t e, p0, p1;
  int32_t slot;  // of the partial sums; -1: the adapter's only chunk
};
// Runs of 16 positions for the products, and chunks for the gradients' sums over tokens: T positions make at most 16 of
// the latter, and adapters of several chunks have at most kAdaptSlots together (count > len gives at most 2 count / len).
constexpr int kAdaptSlots = 32;
inline int adapt_chunk_len(int64_t T) { return T <= 1024 ? 256 : T <= 8192 ? 512 : (int)((T + 511) / 512 * 32); }
inline int64_t adapt_max_chunks(int64_t T, int n) { return 16 + (T < n ? T : n); }
inline int64_t adapt_max_runs(int64_t T, int n) { return T / 16 + (T < n ? T : n); }
struct AdaptOrder {
  int32_t* order;  // [T] token of a position
  int32_t* ad;     // [T] its adapter, -1: none
  int32_t* n_runs;
  AdaptChunk* runs;
  // for the gradients, or nullptr
  int32_t* offsets;  // [n + 1] first position of each adapter, and of the tokens without one
  int32_t* slot0;    // [n] first partial sum of an adapter of several chunks
  int32_t* n_chunks;
  AdaptChunk* chunks;
};
hipError_t launch_adapt_order(const int32_t* ids, int T, int n_ad, const AdaptOrder& out, hipStream_t st);
// Whether s (A x) takes a workgroup for a token and four rows (no order needed) rather than one for a run of 16 positions.
inline bool adapt_few(int64_t T, int R) { return T * R <= 4096; }
// Tokens of a backward pass that needs no order: its products and sums look for their adapters' tokens themselves.
constexpr int kAdaptFewTokens = 64;
// h[p][r] = scale * sum over c of x[order[p]][c] a[ad[p]][r][c] for positions with an adapter; ht, where given, the same as
// [T / 8][R][8]; two such products in one launch
struct AdaptDown {
  struct Part {
    const void* x;  // of the call's type, or fp32
    int64_t ldx;
    int32_t f32, vec_x, C;
    const int32_t* order;
    const void* a;
    int32_t across;  // (few) a lies as [C][R]
    float* h;
    float* ht;
  };
  int32_t T, R, n_ad, parts;
  int32_t few;       // a workgroup for a token and four rows, with ad; else one for each of the order's runs
  int32_t by_token;  // rows of h are tokens
  const int32_t* ad;
  const int32_t* n_runs;  // nullptr: adapter 0 for all
  const AdaptChunk* runs;
  const float* scale;
  Part part[2];
};
hipError_t launch_adapt_down(const AdaptDown& a, int dtype, hipStream_t st);
// out[e] = sum over e's positions of v[p][r] m[p][c]: [n][R][C], or with `rows` [n][C][R]; out NULL: not wanted
struct AdaptOuter {
  struct Part {
    const void* m;  // of the call's type, or fp32
    int64_t ldm;
    int32_t f32, vec_m, C, rows;
    const int32_t* order;  // rows of m, nullptr: m's rows are positions
    const float* v;
    const float* vt;
    float* part;  // [kAdaptSlots][R][C]
    void* out;
  };
  int32_t T, R, n_ad;
  const int32_t* ids;  // without an order: adapter of a token
  AdaptOrder order;    // order.order nullptr: positions are tokens, at most kAdaptFewTokens
  Part part[2];
};
hipError_t launch_adapt_outer(const AdaptOuter& a, int dtype, hipStream_t st);
// out [n][Q][M] = in [n][M][Q] transposed, for the adapters that tokens have; out NULL: not wanted
struct AdaptTranspose {
  struct Part {
    const void* in;
    int32_t M, Q;
    void* out;
  };
  int32_t n_ad;
  const int32_t* offsets;
  Part part[2];
};
hipError_t launch_adapt_transpose(const AdaptTranspose& a, int elem, hipStream_t st);

// ------------------------------------------------------------ gradients' norm (k_clip.hip)
int64_t clip_chunks(const moe_grad* g, int count);
size_t clip_table_bytes(const moe_grad* g, int count);
hipError_t launch_clip_table(const moe_grad* g, int count, void* table, hipStream_t st);
hipError_t launch_clip(const moe_grads& t, float max_norm, float* norm, hipStream_t st);

}  // namespace moe
