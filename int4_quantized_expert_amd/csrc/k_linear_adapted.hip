// k_linear_adapted.hip — y = act(W x + b + s B (A x)) + r with low-rank adapters by token, and the values in front of the
// activation for a backward pass: the kernels of the product with the adapters' second half in their epilogue. The first
// half, s (A x), R values a token, is k_adapt.hip's. For more than a few tokens the tiles work on tokens ordered by adapter.
#define MOE_ADAPTED 1
#define MOE_TRANSPOSED 0
#include "linear_kernels.h"

namespace moe {

namespace {
constexpr int kMixed = 4;
struct AdaptedPlan {
  size_t h, order, ad, n_runs, runs, total;
};
AdaptedPlan adapted_plan(const moe_linear_config& c, const moe_adapters* ad, int64_t T) {
  const size_t R = ad ? ad->rank : 0;
  AdaptedPlan p;
  p.h = up256(linear_ws_bytes(c, T));
  p.order = p.h + up256(T * R * 4);
  p.ad = p.order + up256(T * 4);
  p.n_runs = p.ad + up256(T * 4);
  p.runs = p.n_runs + 256;
  p.total = p.runs + (ad ? up256(sizeof(AdaptChunk) * adapt_max_runs(T, ad->n_adapters)) : 0);
  return p;
}

template <class TX>
hipError_t run(LinearArgs& a, int bits, const moe_adapters* ad, const int32_t* ids, int dtype, void* ws,
               const AdaptedPlan& p, hipStream_t st) {
  char* w = static_cast<char*>(ws);
  const bool few = is_slim(a.T, a.N);
  if (ad) {
    a.h = reinterpret_cast<const float*>(w + p.h);
    a.ab = ad->b;
    a.n_ad = ad->n_adapters;
    a.R = ad->rank;
    a.ad = ids;
    AdaptDown d{};
    d.T = a.T, d.R = a.R, d.n_ad = a.n_ad, d.parts = 1, d.by_token = few, d.few = adapt_few(a.T, a.R);
    d.scale = ad->scale;
    // Few tokens do without an order, and so do any number of one adapter (2,048-token calls save 7 us of 70 to 310), where
    // tokens that have none are computed with it and left out, and not many of a few adapters: 32 neighbours then have at
    // most kMixed of them (191 tokens, rank 8, four adapters, 6144 x 2048 int8: 29.7 us a call, 35.7; 1,500 tokens of four
    // adapters one by one would lose 7 to 14).
    const bool sorted = ids && a.n_ad > 1 && !(adapt_few(a.T, a.R) && (few || a.n_ad <= kMixed));
    const AdaptOrder o{reinterpret_cast<int32_t*>(w + p.order), reinterpret_cast<int32_t*>(w + p.ad),
                       reinterpret_cast<int32_t*>(w + p.n_runs), reinterpret_cast<AdaptChunk*>(w + p.runs)};
    if (sorted) {
      const hipError_t e = launch_adapt_order(ids, a.T, a.n_ad, o, st);
      if (e != hipSuccess) return e;
      d.n_runs = o.n_runs, d.runs = o.runs;
      if (!few) a.order = o.order, a.ad = o.ad;
    }
    d.ad = sorted ? o.ad : ids;
    d.part[0] = {a.x, a.ldx, 0, a.vec_x, a.K, sorted ? o.order : nullptr, ad->a, 0, reinterpret_cast<float*>(w + p.h), nullptr};
    const hipError_t e = launch_adapt_down(d, dtype, st);
    if (e != hipSuccess) return e;
  }
  linear_launch<TX>(a, bits, ws, st);
  return hipGetLastError();
}
}  // namespace

size_t adapted_ws_bytes(const moe_linear_config& c, const moe_adapters* ad, int64_t T) {
  return adapted_plan(c, ad, T).total;
}

hipError_t launch_linear_adapted(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                                 const moe_adapters* ad, const int32_t* ids, const void* x, int64_t ldx, int T, int dtype,
                                 const void* res, int64_t ldr, void* y, int64_t ldy, void* pre, int64_t ldp, void* ws,
                                 hipStream_t st) {
  LinearArgs a = linear_args(c, codes, scales, bias, x, ldx, T, dtype, res, ldr, y, ldy, ws);
  a.pre = pre;
  a.ldp = ldp;
  a.vec_p = reinterpret_cast<uintptr_t>(pre) % (dtype == MOE_DTYPE_F32 ? 16 : 8) == 0 && ldp % 4 == 0;
  const AdaptedPlan p = adapted_plan(c, ad, T);
  const int bits = c.weight_bits == 8 ? 8 : 4;
  if (dtype == MOE_DTYPE_F32) return run<float>(a, bits, ad, ids, dtype, ws, p, st);
  if (dtype == MOE_DTYPE_BF16) return run<bf16_t>(a, bits, ad, ids, dtype, ws, p, st);
  return run<_Float16>(a, bits, ad, ids, dtype, ws, p, st);
}

}  // namespace moe
