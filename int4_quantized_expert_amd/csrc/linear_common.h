// linear_common.h — what the kernels of the products over weight codes share: arguments, activations and codes as fp16,
// the epilogue.
//
// Both operands go to the matrix cores as fp16, without loss:
//  - a code (at most 8 bits) is an integer that fp16 holds exactly; its scale multiplies the fp32 sum.
//  - an activation is multiplied by a power of two per token, such that the token's largest lies in [2^14, 2^15).
//    fp16 then holds every bf16 value down to 2^-31 of the largest exactly, and any smaller one to 2^-38 of the
//    largest. fp32 values are split, v = hi + lo, both fp16: what is lost is below 2^-23 of the value (or 2^-38 of
//    the token's largest). fp16 values are taken as they are.
// Products are exact in fp32, sums are fp32.
//
// Unpacking a word of eight nibbles: the nibble, moved to 0..15 by flipping its top bit, is put into the low (or
// next) mantissa bits of 1024.0; a packed subtraction (or multiply-add by 1/16) leaves the code. That gives the
// element order 0 4 1 5 2 6 3 7, in which the activations are stored too.
//
// A source that includes this says first what its kernels do besides: MOE_ADAPTED, low-rank adapters (and saving the
// values in front of the activation) in the epilogue; MOE_TRANSPOSED, sums over the weight rows (linear_kernels.h).
#pragma once

#include <algorithm>

#include "linear_types.h"

namespace moe {

namespace {

constexpr bool kAdapted = MOE_ADAPTED, kTransposed = MOE_TRANSPOSED;

struct LinearArgs {
  int32_t T, N, K, nb, nbp;  // tokens, weight rows, columns, 32-blocks of a row, blocks padded to a multiple of 2
  int32_t half;              // rows of the gate part (SwiGLU), else 0
  int32_t vec_x;             // rows of x start on 16-byte boundaries
  int32_t vec_r, vec_y;      // rows of the residual and of y on boundaries of four elements
  int32_t act, gshift;       // gshift: log2(group / 32), -1 for one scale a row
  const uint8_t* codes;
  const float* scales;
  const float* bias;
  const void* x;
  const void* res;
  void* y;
  int64_t ldx, ldr, ldy;
  _Float16* xh;  // [T/32][nbp][4 slices][32 tokens][8]: activations as fp16, and
  _Float16* xl;  // their rest (fp32 activations only), same order
  int32_t* sh;   // [T] power of two that token t was multiplied by

  // kAdapted. Tiles work on positions: tokens in the order of their adapters, so that few of a tile's tokens differ in it.
  const int32_t* order;  // [T] token of a position, nullptr where positions are tokens
  const int32_t* ad;     // [T] adapter of a position (outside 0 .. n_ad - 1: none), nullptr: adapter 0 for all
  const float* h;        // [T][R] of a position: adapter scale times (A x); nullptr: no adapters
  const void* ab;        // [n_ad][N][R]
  int32_t n_ad, R;
  void* pre;  // values in front of the activation, rows ldp apart, or nullptr
  int64_t ldp;
  int32_t vec_p;

  // kTransposed with group scales: those of each row over the power of two that was multiplied into the activations,
  // [rows / 64][groups][64] as fp16 in the codes' order: for bf16 calls the scale, for fp16 and fp32 calls eight bits of it,
  // and gs_low further on the rest
  const _Float16* gs;
  int64_t gs_low;
};

__device__ __forceinline__ int token_of(const LinearArgs& a, int p) { return kAdapted && a.order ? a.order[p] : p; }
__device__ __forceinline__ int adapter_of(const LinearArgs& a, int p) {
  const int id = a.ad ? a.ad[p] : 0;
  return (uint32_t)id < (uint32_t)a.n_ad ? id : -1;
}

// ------------------------------------------------------------ activations to fp16
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
// Largest magnitudes: the bits without the sign, compared as integers (infinity and NaN come out on top). bf16: two in
// one word.
template <class TX>
__device__ __forceinline__ void amax8(const Granule<TX>& d, uint32_t& m) {
#pragma unroll
  for (int i = 0; i < (int)(2 * sizeof(TX)); ++i) {
    if (sizeof(TX) == 4) {
      m = max(m, d.w[i] & 0x7FFFFFFFu);
    } else {
      const us2 v = __builtin_bit_cast(us2, d.w[i] & 0x7FFF7FFFu);
      m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, m), v));
    }
  }
}
template <class TX>
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) {
  return sizeof(TX) == 4 ? m : max(m << 16, m & 0xFFFF0000u);
}
// power of two for the largest magnitude: 0 where it is zero, infinite or NaN
__device__ __forceinline__ int scale_shift(uint32_t amax) {
  return amax > 0 && amax < 0x7F800000u ? 14 - ((int)(amax >> 23) - 127) : 0;
}
// Element pairs (0 4) (1 5) (2 6) (3 7) as fp16. finite: the token holds neither infinity nor NaN; otherwise its
// finite values are only kept finite.
template <class TX>
__device__ __forceinline__ void convert8(const Granule<TX>& d, int sh, bool finite, h8& hi, h8& lo) {
  if constexpr (std::is_same<TX, _Float16>::value) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[2 * i] = __builtin_amdgcn_perm(d.w[i + 2], d.w[i], 0x05040100u);
      o[2 * i + 1] = __builtin_amdgcn_perm(d.w[i + 2], d.w[i], 0x07060302u);
    }
    __builtin_memcpy(&hi, o, 16);
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (i >> 1) + 4 * (i & 1);
      uint32_t u;
      if (sizeof(TX) == 4) u = d.w[e & (2 * sizeof(TX) - 1)];
      else u = e & 1 ? d.w[e >> 1] & 0xFFFF0000u : d.w[e >> 1] << 16;
      v[i] = ldexpf(__uint_as_float(u), sh);
    }
    if (!finite)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (fabsf(v[i]) < INFINITY) v[i] = fminf(fmaxf(v[i], -65504.0f), 65504.0f);
    if constexpr (sizeof(TX) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hi[i] = (_Float16)v[i];
        lo[i] = (_Float16)(v[i] - (float)hi[i]);
      }
      if (!finite)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(fabsf(v[i]) < INFINITY)) lo[i] = (_Float16)0.0f;
    } else {  // a bf16 value fits, or is far below the largest: rounding toward zero serves
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(v[2 * i], v[2 * i + 1]));
      __builtin_memcpy(&hi, o, 16);
    }
  }
}

// ------------------------------------------------------------ codes to fp16
__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }
__device__ __forceinline__ h8 join(h2 a, h2 b, h2 c, h2 d) {
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// eight nibbles
__device__ __forceinline__ h8 codes_h8(uint32_t w) {
  const uint32_t u = w ^ 0x88888888u, v = u >> 8;
  const h2 off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
  const h2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f}, off16 = {(_Float16)-72.0f, (_Float16)-72.0f};
  const h2 p0 = as_h2((u & 0x000F000Fu) | 0x64006400u) + off;
  const h2 p1 = __builtin_elementwise_fma(as_h2((u & 0x00F000F0u) | 0x64006400u), sixteenth, off16);
  const h2 p2 = as_h2((v & 0x000F000Fu) | 0x64006400u) + off;
  const h2 p3 = __builtin_elementwise_fma(as_h2((v & 0x00F000F0u) | 0x64006400u), sixteenth, off16);
  return join(p0, p1, p2, p3);
}
// eight bytes, stored even elements first
__device__ __forceinline__ h8 codes_h8(uint32_t even, uint32_t odd) {
  const uint32_t u = even ^ 0x80808080u, v = odd ^ 0x80808080u;
  const h2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  return join(as_h2((u & 0x00FF00FFu) | 0x64006400u) + off, as_h2((v & 0x00FF00FFu) | 0x64006400u) + off,
              as_h2((u >> 8 & 0x00FF00FFu) | 0x64006400u) + off, as_h2((v >> 8 & 0x00FF00FFu) | 0x64006400u) + off);
}

// ------------------------------------------------------------ epilogue
__device__ __forceinline__ float activate(float v, int act) {
  float s, miss;
  switch (act) {
    case MOE_ACT_RELU: return v <= 0.0f ? 0.0f : v;  // NaN stays
    case MOE_ACT_SILU: sigmoid2(v, s, miss); return v * s;
    case MOE_ACT_GELU: return 0.5f * v * erfcf(v * -0.707106781f);
    case MOE_ACT_GELU_TANH: sigmoid2(1.59576912f * v * fmaf(0.044715f * v, v, 1.0f), s, miss); return v * s;
    default: return v;
  }
}
// What an adapter adds to output `row` of position p: a dot product of R terms, for few tokens.
template <class TX>
__device__ __forceinline__ float adapter_dot(const LinearArgs& a, int p, int id, int row) {
  const TX* b = static_cast<const TX*>(a.ab) + ((size_t)id * a.N + row) * a.R;
  const float* h = a.h + (size_t)p * a.R;
  float v = 0.0f;
  for (int r = 0; r < a.R; r += 8) {
    Granule<TX> d;
    load8(b + r, true, d);
    const f8v w = granule_f32<TX>(d);
#pragma unroll
    for (int i = 0; i < 8; ++i) v = fmaf(h[r + i], w[i], v);
  }
  return v;
}

// Few tokens: positions are tokens.
template <class TX>
__device__ __forceinline__ void finish(const LinearArgs& a, int t, int col, float v, float up) {
  if constexpr (kAdapted) {
    const int id = a.h ? adapter_of(a, t) : -1;
    if (id >= 0) {
      v += adapter_dot<TX>(a, t, id, col);
      if (a.act == MOE_ACT_SWIGLU) up += adapter_dot<TX>(a, t, id, a.half + col);
    }
  }
  if (a.bias) v += a.bias[col];
  if (a.act == MOE_ACT_SWIGLU && a.bias) up += a.bias[a.half + col];
  if constexpr (kAdapted)
    if (a.pre) {
      TX* p = static_cast<TX*>(a.pre) + (size_t)t * a.ldp + col;
      *p = from_f32<TX>(v);
      if (a.act == MOE_ACT_SWIGLU) p[a.half] = from_f32<TX>(up);
    }
  if (a.act == MOE_ACT_SWIGLU) {
    float s, miss;
    sigmoid2(v, s, miss);
    v = v * s * up;
  } else {
    v = activate(v, a.act);
  }
  if (a.res) v += to_f32<TX>(static_cast<const TX*>(a.res)[(size_t)t * a.ldr + col]);
  static_cast<TX*>(a.y)[(size_t)t * a.ldy + col] = from_f32<TX>(v);
}

// Four neighbouring outputs of token t, already converted back by 2^back.
template <class TX>
__device__ __forceinline__ void finish4(const LinearArgs& a, int t, int col, int back, const float* gate, const float* up) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ldexpf(gate[i], back);
  if (a.bias)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += a.bias[col + i];
  float zs[4], ups[4];  // as they are in front of the activation
  if (kAdapted)
#pragma unroll
    for (int i = 0; i < 4; ++i) zs[i] = v[i];
  if (a.act == MOE_ACT_SWIGLU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s, miss, u = ldexpf(up[i], back);
      if (a.bias) u += a.bias[a.half + col + i];
      if (kAdapted) ups[i] = u;
      sigmoid2(v[i], s, miss);
      v[i] = v[i] * s * u;
    }
  } else if (a.act != MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = activate(v[i], a.act);
  }
  struct alignas(4 * sizeof(TX)) Four {
    TX v[4];
  };
  if (kAdapted && a.pre) {
    auto save = [&](TX* p, const float* z) __attribute__((always_inline)) {
      Four o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o.v[i] = from_f32<TX>(z[i]);
      if (a.vec_p) *reinterpret_cast<Four*>(p) = o;
      else
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = o.v[i];
    };
    TX* p = static_cast<TX*>(a.pre) + (size_t)t * a.ldp + col;
    save(p, zs);
    if (a.act == MOE_ACT_SWIGLU) save(p + a.half, ups);
  }
  if (a.res) {
    const TX* p = static_cast<const TX*>(a.res) + (size_t)t * a.ldr + col;
    Four r;
    if (a.vec_r) r = *reinterpret_cast<const Four*>(p);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = p[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += to_f32<TX>(r.v[i]);
  }
  TX* p = static_cast<TX*>(a.y) + (size_t)t * a.ldy + col;
  Four o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.v[i] = from_f32<TX>(v[i]);
  if (a.vec_y) *reinterpret_cast<Four*>(p) = o;
  else
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = o.v[i];
}

// ------------------------------------------------------------ workspace of the tiles' activations
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct LinearPlan {
  size_t xh, xl, sh, total;
};
inline LinearPlan linear_plan(int K, int64_t T) {
  LinearPlan p;
  const size_t nbp = (size_t)((K / 32 + 1) & ~1), tp = (size_t)((T + 31) / 32) * 32;
  const size_t x = up256(tp * nbp * 32 * 2);
  p.xh = 0;
  p.xl = x;
  p.sh = 2 * x;
  p.total = p.sh + up256((size_t)T * 4);
  return p;
}

// log2(group / 32), -1 for one scale a row
inline int group_shift(const moe_linear_config& c) {
  int s = -1;
  if (c.group_size > 0)
    for (s = 0; (32 << s) < c.group_size;) ++s;
  return s;
}

}  // namespace

}  // namespace moe
