// k_linear.hip — y = act(W x + b) + r over the library's row-tiled int4 / int8 codes, activations in fp32, bf16 or
// fp16 and not quantized.
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
#include <algorithm>
#include <type_traits>

#include "moe_float.h"
#include "moe_ops.h"

namespace moe {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef int i4v __attribute__((ext_vector_type(4)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

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
};

// ------------------------------------------------------------ activations to fp16
// A granule: eight neighbouring elements of a token as they lie in memory.
template <class TX>
struct Granule {
  uint32_t w[2 * sizeof(TX)];
};
// vec: the rows of x start on 16-byte boundaries
template <class TX>
__device__ __forceinline__ void load8(const TX* p, bool vec, Granule<TX>& d) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(TX) / 2; ++i) {
      const u4v v = reinterpret_cast<const u4v*>(p)[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) d.w[4 * i + j] = v[j];
    }
  } else {
    TX v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
    __builtin_memcpy(&d, v, sizeof(d));
  }
}
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

// ------------------------------------------------------------ activations to fp16 in tile order
// One workgroup takes 8 tokens: thread = (token tid % 8, granule of 8 elements tid / 8), so 8 neighbouring threads
// write 128 contiguous bytes and each token is read in runs of 128 granules. Up to 8 granules a thread (8192 columns)
// stay in registers between the search for the largest and the conversion; of longer rows the rest is read twice.
constexpr int kPrepLanes = 128, kPrepRounds = 8;
template <class TX>
__global__ __launch_bounds__(8 * kPrepLanes) void k_linear_x(LinearArgs a) {
  __shared__ uint32_t s_max[16][8];
  const int tk = threadIdx.x & 7, g0 = threadIdx.x >> 3;
  const int t = blockIdx.x * 8 + tk;
  const bool in = t < a.T;
  const TX* row = static_cast<const TX*>(a.x) + (size_t)(in ? t : 0) * a.ldx;
  const int ng = in ? a.K / 8 : 0;
  Granule<TX> raw[kPrepRounds];
#pragma unroll
  for (int k = 0; k < kPrepRounds; ++k)
    if (g0 + k * kPrepLanes < ng) load8(row + (g0 + k * kPrepLanes) * 8, a.vec_x, raw[k]);
  int sh = 0;
  bool finite = true;
  if constexpr (!std::is_same<TX, _Float16>::value) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kPrepRounds; ++k)
      if (g0 + k * kPrepLanes < ng) amax8<TX>(raw[k], m);
    for (int g = g0 + kPrepRounds * kPrepLanes; g < ng; g += kPrepLanes) {
      Granule<TX> v;
      load8(row + g * 8, a.vec_x, v);
      amax8<TX>(v, m);
    }
    m = amax_bits<TX>(m);
#pragma unroll
    for (int o = 8; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((threadIdx.x & 63) < 8) s_max[threadIdx.x >> 6][tk] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, s_max[i][tk]);
    finite = m < 0x7F800000u;
    sh = scale_shift(m);
  }
  if (in && g0 == 0) a.sh[t] = sh;
  const size_t base = (size_t)(t >> 5) * a.nbp * 1024 + (size_t)(t & 31) * 8;
  auto store = [&](int g, const Granule<TX>& v) __attribute__((always_inline)) {
    h8 hi = {}, lo = {};
    if (g < ng) convert8<TX>(v, sh, finite, hi, lo);
    const size_t at = base + (size_t)g * 256;  // g = block * 4 + slice
    *reinterpret_cast<h8*>(a.xh + at) = hi;
    if (std::is_same<TX, float>::value) *reinterpret_cast<h8*>(a.xl + at) = lo;
  };
#pragma unroll
  for (int k = 0; k < kPrepRounds; ++k)
    if (g0 + k * kPrepLanes < a.nbp * 4) store(g0 + k * kPrepLanes, raw[k]);
  for (int g = g0 + kPrepRounds * kPrepLanes; g < a.nbp * 4; g += kPrepLanes) {
    Granule<TX> v = {};
    if (g < ng) load8(row + g * 8, a.vec_x, v);
    store(g, v);
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
template <class TX>
__device__ __forceinline__ void finish(const LinearArgs& a, int t, int col, float v, float up) {
  if (a.bias) v += a.bias[col];
  if (a.act == MOE_ACT_SWIGLU) {
    float s, miss;
    if (a.bias) up += a.bias[a.half + col];
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
  if (a.act == MOE_ACT_SWIGLU) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s, miss, u = ldexpf(up[i], back);
      if (a.bias) u += a.bias[a.half + col + i];
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

// ------------------------------------------------------------ product
// A wavefront multiplies 32*TT tokens by two fragments of 32 weight rows (64 consecutive rows; with SwiGLU 32 gate
// rows and the 32 up rows that go with them) with v_mfma_f32_32x32x16_f16; RW wavefronts of a workgroup take the same
// tokens. A code fragment costs 10 vector instructions to unpack and serves TT matrix instructions of 8 passes: with
// TT = 4 the unpacking fits between them, with TT = 1 it takes the longer time. 2,048 tokens 12288 x 6144 with SwiGLU:
// 181 us for the 512 whole tiles and 99 for the rest, 1.14 PFLOP/s and 1.04, matrix instructions busy for 61% and 52%;
// 191 tokens 6144 x 2048 int8 at TT = 1: 20.5 us, 18%. fp32 at TT = 1, 1,001 tokens 6144 x 4096: 119 us in the median,
// 108 at best, 0.85 to 0.94 PFLOP/s of halves, 51%.
// The activations of a step (two blocks of columns) pass through LDS in two buffers: the next step's are loaded to
// registers while this one is multiplied. Each wavefront reads its own codes from memory into registers, also a step
// ahead.
// Lane l: token / weight row l % 32, half g = l / 32 of a block. Result: weight row l % 32, tokens
// 8*(i/4) + 4*g + i%4. GSH: -1 one scale a row, 0 groups of one block, 1 groups of two blocks or more.
constexpr int kOutRow = 260;  // floats of a token's row of results in LDS: 256 and a shift of four banks
template <class TX, int TT, int RW, int KW>
constexpr size_t tile_lds() {
  return std::max<size_t>({(size_t)KW * 2 * TT * (std::is_same<TX, float>::value ? 2 : 1) * 4096,
                           (size_t)(KW / 2) * RW * 8 * 1024, (size_t)16 * kOutRow * 4});
}

// KW groups of RW wavefronts: a group's wavefronts take 64 rows each, from wavefront tile wt0 on, the groups share the
// columns.
template <class TX, int TT, int W, int GSH, int RW, int KW>
__device__ __forceinline__ void tile_run(const LinearArgs& a, int wt0, int t0, char* s_mem) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1;
  constexpr int kStep = NX * TT * 2048;  // halfs of a step: [NX][TT][2 blocks][4 slices][32][8]
  // values that are equal in a wavefront are made so for the compiler: addresses are then a scalar base and a lane's
  // constant offset, without vector arithmetic in the loop
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kLanes = 64 * RW;  // of a group
  const int lane = threadIdx.x & 63, wave = wv % RW, r = lane & 31, g = lane >> 5;
  const int kw = wv / RW, tid = threadIdx.x % kLanes;
  auto s_x = reinterpret_cast<_Float16(*)[kStep]>(s_mem) + kw * 2;
  const int steps = (a.nbp / 2 + KW - 1) / KW, p0 = min(kw * steps, a.nbp / 2), p1 = min(p0 + steps, a.nbp / 2);
  const int cols = a.half ? a.half / 32 : a.N / 64;  // wavefront tiles over the outputs
  const int wtc = min(wt0 + wave, cols - 1);
  int first[2];  // first weight row of a fragment
  first[0] = a.half ? wtc * 32 : wtc * 64;
  first[1] = a.half ? a.half + wtc * 32 : wtc * 64 + 32;
  const uint8_t* src[2];
  const float* ssrc[2];
  const int groups = GSH >= 0 ? a.nb >> a.gshift : 0;
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    src[f] = a.codes + tbw_off<W>(first[f] / 64, 0, a.nb) + (size_t)(first[f] % 64) * (4 * W);
    ssrc[f] = a.scales + (GSH >= 0 ? (size_t)(first[f] / 64) * groups * 64 + first[f] % 64 : (size_t)first[f]);
  }
  const uint32_t off0 = r * (4 * W), off1 = off0 + g * (uint32_t)kTileBlock<W>;
  // this workgroup's [2 blocks][4 slices][32][8] chunks, 16 bytes a lane
  const _Float16* xsrc[TT];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) xsrc[tt] = a.xh + (size_t)min(t0 / 32 + tt, (a.T - 1) / 32) * a.nbp * 1024;
  const size_t low = a.xl - a.xh;
  constexpr int kScales = GSH == 0 ? 2 : 1;
  constexpr int kXs = 4 / RW;  // 16-byte loads of a lane and chunk
  u4v xn[NX][TT][kXs];  // activations and
  uint32_t wn[2][W];  // codes of the next step
  float sn[2][kScales], sc[2][kScales];
  h8 wf[2][2][2];  // this step's fragments: [block][m][fragment]
  auto fetch_x = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NX; ++n)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int j = 0; j < kXs; ++j)
          xn[n][tt][j] =
              *reinterpret_cast<const u4v*>(xsrc[tt] + n * low + (size_t)p * 2048 + (uint32_t)((j * kLanes + tid) * 8));
  };
  auto fetch_w = [&](int p) __attribute__((always_inline)) {
    const uint32_t off = 2 * p + 1 < a.nb ? off1 : off0;  // past the last block the activations are zero
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const u4v* q = reinterpret_cast<const u4v*>(src[f] + (size_t)p * (2 * kTileBlock<W>) + off);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const u4v v = q[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) wn[f][4 * i + j] = v[j];
      }
      if constexpr (GSH >= 0)
#pragma unroll
        for (int i = 0; i < kScales; ++i)
          sn[f][i] = ssrc[f][(size_t)(min(2 * p + i, a.nb - 1) >> a.gshift) * 64 + (uint32_t)r];
    }
  };
  auto unpack = [&](h8 (&d)[2][2][2], float (&ds)[2][kScales]) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      if constexpr (GSH >= 0)
#pragma unroll
        for (int j = 0; j < kScales; ++j) ds[f][j] = sn[f][j];
      uint32_t w[W];
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = wn[f][j];
      // half g of both blocks instead of all of block 2p + g
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        const auto sw = __builtin_amdgcn_permlane32_swap(w[j], w[j + W / 2], false, false);
        w[j] = sw[0];
        w[j + W / 2] = sw[1];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if constexpr (W == 4) d[h][m][f] = codes_h8(w[2 * h + m]);
          else d[h][m][f] = codes_h8(w[4 * h + 2 * m], w[4 * h + 2 * m + 1]);
        }
    }
  };
  auto put = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < NX; ++n)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int j = 0; j < kXs; ++j)
          *reinterpret_cast<u4v*>(&s_x[buf][((n * TT + tt) * 256 + j * kLanes + tid) * 8]) = xn[n][tt][j];
  };
  f16v acc[TT][2];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[tt][f][i] = 0.0f;
  auto multiply = [&](const _Float16* x) __attribute__((always_inline)) {
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      f16v c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NX; ++n) {
            const h8 xf = *reinterpret_cast<const h8*>(x + (((n * TT + tt) * 2 + h) * 4 + 2 * g + m) * 256 + r * 8);
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              if constexpr (GSH < 0) {
                acc[tt][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, wf[h][m][f], acc[tt][f], 0, 0, 0);
              } else {
                const bool first = m == 0 && n == 0 && (GSH == 0 || h == 0);
                f16v zero;
#pragma unroll
                for (int j = 0; j < 16; ++j) zero[j] = 0.0f;
                c[f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, wf[h][m][f], first ? zero : c[f], 0, 0, 0);
              }
            }
          }
        if constexpr (GSH >= 0)
          if (GSH == 0 || h == 1)
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[tt][f][j] = fmaf(c[f][j], sc[f][h & (kScales - 1)], acc[tt][f][j]);
      }
    }
  };
  if (p0 < p1) {
    fetch_x(p0);
    fetch_w(p0);
    put(0);
  }
  if constexpr (TT == 4) {
    // The next step's codes are unpacked between this step's matrix instructions. Past the last step the fetches repeat
    // it and their results are not used: the body has no branch, which would keep the two apart. 8,192 tokens
    // 12288 x 6144: 1,002 us with the unpacking in front, 968 so; with fewer matrix instructions a step it was slower.
    unpack(wf, sc);
    fetch_x(min(p0 + 1, p1 - 1));
    fetch_w(min(p0 + 1, p1 - 1));
    __syncthreads();
    for (int i = 0; i < steps; ++i, __syncthreads()) {
      const int p = p0 + i;
      if (KW > 1 && p >= p1) continue;  // a group with fewer columns
      h8 wl[2][2][2];
      float sl[2][kScales];
      unpack(wl, sl);
      fetch_w(min(p + 2, p1 - 1));
      put((i + 1) & 1);
      fetch_x(min(p + 2, p1 - 1));
      multiply(s_x[i & 1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int f = 0; f < 2; ++f) wf[h][m][f] = wl[h][m][f];
    }
  } else {
    // 64 tokens and two groups of columns: the second group, the other wavefront of each SIMD, unpacks the next step's
    // codes behind its matrix instructions, so that between two barriers one's unpacking runs beside the other's products
    // (400 tokens, 8192 x 4096: 45.7 us, 49.4 with both in front). With 32 tokens it was up to 5% slower, with a scale a
    // block it takes too many registers, and reading codes two or three steps ahead gained nothing.
    const bool late = TT == 2 && KW == 2 && GSH != 0 && kw > 0;
    if (late && p0 < p1) {
      unpack(wf, sc);
      fetch_w(min(p0 + 1, p1 - 1));
    }
    __syncthreads();
    for (int i = 0; i < steps; ++i, __syncthreads()) {
      const int p = p0 + i;
      if (KW > 1 && p >= p1) continue;  // a group with fewer columns
      const bool more = p + 1 < p1;
      if (!late) unpack(wf, sc);
      if (more) {
        fetch_x(p + 1);
        if (!late) fetch_w(p + 1);
      }
      multiply(s_x[i & 1]);
      if (more) {
        put((i + 1) & 1);
        if (late) {
          unpack(wf, sc);
          fetch_w(min(p + 2, p1 - 1));
        }
      }
    }
  }
  // the groups' sums: the upper half to the lower until one is left, 32 tokens at a time
#pragma unroll
  for (int k = KW / 2; k > 0; k >>= 1) {
    float* s = reinterpret_cast<float*>(s_mem);  // [group][32][kLanes]
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      if (kw >= k && kw < 2 * k)
#pragma unroll
        for (int i = 0; i < 32; ++i) s[((kw - k) * 32 + i) * kLanes + tid] = acc[tt][i >> 4][i & 15];
      __syncthreads();
      if (kw < k)
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[tt][i >> 4][i & 15] += s[(kw * 32 + i) * kLanes + tid];
      __syncthreads();
    }
  }
  float rs[2] = {1.0f, 1.0f};
  if (GSH < 0) rs[0] = ssrc[0][r], rs[1] = ssrc[1][r];
  // results through LDS, 16 tokens at a time, so that they are finished and stored four neighbours a lane
  float* s_out = reinterpret_cast<float*>(s_mem);
  const int at0 = a.half ? wave * 32 + r : wave * 64 + r, at1 = 32 * (a.half ? RW : 1) + at0;
  const int quads = (a.half ? 8 : 16) * RW, col0 = wt0 * (a.half ? 32 : 64), out = a.half ? a.half : a.N;
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      __syncthreads();
      if (kw == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tk = 8 * (i >> 2) + 4 * g + (i & 3);
          s_out[tk * kOutRow + at0] = acc[tt][0][8 * hh + i] * rs[0];
          s_out[tk * kOutRow + at1] = acc[tt][1][8 * hh + i] * rs[1];
        }
      __syncthreads();
      for (int k = threadIdx.x; k < 16 * quads; k += kLanes * KW) {
        const int tk = k / quads, c = k % quads * 4, t = t0 + 32 * tt + 16 * hh + tk;
        if (t < a.T && col0 + c < out)
          finish4<TX>(a, t, col0 + c, -a.sh[t], s_out + tk * kOutRow + c,
                      s_out + tk * kOutRow + 32 * RW + c);
      }
    }
}

// Tiles of 32*BT tokens by 256 rows, numbered so that 8 row tiles are walked by all token tiles; a launch takes `count`
// of them from `first` on, each cut into BT / TT by 4 / RW workgroups of 32*TT tokens and 64*RW rows. Workgroups go to
// the eight dies in turn: die d takes the d-th eighth of a launch, so that what a die works on at a time shares its
// cache.
constexpr int kTileRowGroup = 8, kDies = 8;
template <class TX, int GSH>
constexpr int base_frags() {  // 128 tokens need too many registers with two halves of them or a second set of sums
  return std::is_same<TX, float>::value || GSH >= 0 ? 2 : 4;
}

template <class TX, int TT, int W, int GSH, int RW, int KW>
__global__ __launch_bounds__(64 * RW * KW, RW * KW == 16 ? 4 : 2) void k_linear_tile(LinearArgs a, int row_tiles,
                                                                                     int tok_tiles, int first,
                                                                                     int count) {
  constexpr int BT = base_frags<TX, GSH>(), kToks = BT / TT, kRows = 4 / RW;  // the cut of a tile
  __shared__ __align__(16) char s_mem[tile_lds<TX, TT, RW, KW>()];
  const int n = count * kToks * kRows, d = blockIdx.x % kDies, q = n / kDies, m = n % kDies;
  const int k = d * q + min(d, m) + blockIdx.x / kDies, id = first + k / (kToks * kRows);
  const int group = id / (kTileRowGroup * tok_tiles), in_group = id - group * kTileRowGroup * tok_tiles;
  const int rows_in = min(kTileRowGroup, row_tiles - group * kTileRowGroup);
  const int t0 = in_group / rows_in * 32 * BT + k % kToks * 32 * TT;
  const int wt0 = (group * kTileRowGroup + in_group % rows_in) * 4 + k / kToks % kRows * RW;
  if (t0 < a.T && wt0 * (a.half ? 32 : 64) < (a.half ? a.half : a.N)) tile_run<TX, TT, W, GSH, RW, KW>(a, wt0, t0, s_mem);
}

// ------------------------------------------------------------ few tokens: product
// Reading the codes is what counts: all of them are in flight at once. v_mfma_f32_16x16x32_f16 multiplies 16 tokens by
// fragments of 16 weight rows, F of them in a wavefront (with SwiGLU 16 gate rows and the 16 up rows that go with
// them).
// Codes: lane (row r = l % 16, g = l / 16) loads the 16 bytes (int8: 32) of its row in block 4q + g. With one scale a
// row, instruction i then takes slice i of the four blocks; with group scales a 4 x 4 transposition over the lane
// groups leaves the lane slice g of each block, so that one instruction covers one block and scales are applied
// between blocks.
// Activations are converted in LDS, order [blocks][4 slices][tokens][8], each token multiplied by a power of two of its
// own. Their loads are issued ahead of the codes' (loads return in order) and stay in registers while the largest is
// found.
typedef float f4v __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void transpose4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  auto s = __builtin_amdgcn_permlane32_swap(a, c, false, false);
  a = s[0], c = s[1];
  s = __builtin_amdgcn_permlane32_swap(b, d, false, false);
  b = s[0], d = s[1];
  s = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = s[0], b = s[1];
  s = __builtin_amdgcn_permlane16_swap(c, d, false, false);
  c = s[0], d = s[1];
}

// One quad of blocks of a fragment: codes and scales. GSH: -1 one scale a row, else log2(group / 32), at most 2 (a
// larger group has one scale for the quad too).
template <int W, int GSH>
struct Quad {
  static constexpr int kScales = GSH < 0 ? 1 : 4 >> GSH;
  uint32_t w[W];
  float s[kScales];
};

// A wavefront's weight rows.
template <int W, int GSH, int F>
struct Rows {
  int row[F];
  const uint8_t* src[F];
  const float* scale[F];
  int g, nb, gshift;

  // output columns out0 .. of the F fragments
  __device__ __forceinline__ Rows(const LinearArgs& a, int out0, int lane) : g(lane >> 4), nb(a.nb), gshift(a.gshift) {
    const int r = lane & 15, groups = GSH >= 0 ? a.nb >> a.gshift : 0;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      row[f] = a.half ? f * a.half + min(out0 + r, a.half - 1) : min(out0 + 16 * f + r, a.N - 1);
      src[f] = a.codes + tbw_off<W>(row[f] / 64, 0, a.nb) + (size_t)(row[f] % 64) * (4 * W);
      scale[f] = a.scales + (GSH >= 0 ? (size_t)(row[f] / 64) * groups * 64 + row[f] % 64 : (size_t)row[f]);
    }
  }
  // blocks b .. b + 3; past the last block the activations are zero, so any codes will do
  __device__ __forceinline__ void load(Quad<W, GSH> (&d)[F], int b) const {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const u4v* p = reinterpret_cast<const u4v*>(src[f] + (size_t)min(b + g, nb - 1) * kTileBlock<W>);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const u4v v = __builtin_nontemporal_load(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[f].w[4 * i + j] = v[j];
      }
      if constexpr (GSH >= 0)
#pragma unroll
        for (int i = 0; i < Quad<W, GSH>::kScales; ++i)
          d[f].s[i] = scale[f][(size_t)(min(b + (i << GSH), nb - 1) >> gshift) * 64];
    }
  }
};

// acc += quad times activations. x: LDS of the quad's first block; token fragment n and half v start at
// (v * NT + n) * stride halfs; a block has 4 slices of TOK tokens of 8 halfs; rt the lane's token.
template <int NX, int NT, int TOK, int W, int GSH, int F>
__device__ __forceinline__ void multiply_quad(Quad<W, GSH> (&d)[F], const _Float16* x, int stride, int rt, int g,
                                              f4v (&acc)[NT][F]) {
  if constexpr (GSH >= 0)
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (W == 4) {
        transpose4(d[f].w[0], d[f].w[1], d[f].w[2], d[f].w[3]);
      } else {  // slice j: words 2j and 2j + 1
        transpose4(d[f].w[0], d[f].w[2], d[f].w[4], d[f].w[6]);
        transpose4(d[f].w[1], d[f].w[3], d[f].w[5], d[f].w[7]);
      }
    }
  f4v c[NT][F];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool first = GSH == 0 || (GSH == 1 && (i & 1) == 0) || i == 0;
    const bool last = GSH == 0 || (GSH == 1 && (i & 1) == 1) || i == 3;
    h8 wf[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (W == 4) wf[f] = codes_h8(d[f].w[i]);
      else wf[f] = codes_h8(d[f].w[2 * i], d[f].w[2 * i + 1]);
    }
    const int slice = GSH < 0 ? g * 4 + i : i * 4 + g;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int v = 0; v < NX; ++v) {
        const h8 xf = *reinterpret_cast<const h8*>(x + (v * NT + n) * stride + (slice * TOK + rt) * 8);
#pragma unroll
        for (int f = 0; f < F; ++f) {
          if (GSH < 0) {
            acc[n][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xf, wf[f], acc[n][f], 0, 0, 0);
          } else {
            const f4v zero = {0.0f, 0.0f, 0.0f, 0.0f};
            c[n][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xf, wf[f], first && v == 0 ? zero : c[n][f], 0, 0, 0);
          }
        }
      }
    if (GSH >= 0 && last) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[n][f][j] = fmaf(c[n][f][j], d[f].s[(i >> (GSH < 0 ? 0 : GSH)) & (Quad<W, GSH>::kScales - 1)], acc[n][f][j]);
    }
  }
}

// Orders a wavefront's LDS writes before its later reads of other lanes' data.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Up to 4 tokens (TOK 1 or 4): a workgroup finishes 16 rows (with SwiGLU 16 gate and 16 up rows) in one launch. Its
// wavefronts share the columns; each converts its own columns of the tokens, with a power of two of its own, and waits
// for no other before the sum. Bound by the latency of one pass over the codes: 1 token, 6144 x 6144 int4, 8.4 us on
// codes that come from HBM (19 MB: 3.6 to 4.0 by a plain read), 10.4 in the form below; 4 tokens 9.9 and 11.2; 4096 x
// 2048 4.5 and 7.6. int8 6144 x 6144 12.4, SwiGLU 12288 x 6144 11.8. Of the 128 registers of four wavefronts a SIMD some
// forms spill: with SwiGLU int8 (fp32, fp16) and fp16 in groups of 32, 12 to 30; fp16 in groups of 64 with SwiGLU, bf16
// int8 and fp16 heads in groups of 32, 2 to 8.
// TURNS: rows for more than three times the workgroups that run at a time, a head's: a workgroup converts once and takes
// its share of the rows in turns, the next rows' codes on their way while it finishes some. 32768 x 6144, 1 token: 24.0
// us, 27.4 without; 65536 x 4096 g64, 3 tokens: 40.3 and 48.3; three turns (16448 rows) 18.0 and 16.9, two of SwiGLU (24576
// rows) 19.1 and 17.9.
constexpr int kTinyWaves = 8;
constexpr int kTinyGroups = 512;  // workgroups at most: two a compute unit
constexpr int tiny_rounds(size_t size) { return size == 4 ? 4 : 8; }  // granules of 32 bytes or 16 that a lane converts

// One scale a row is taken apart into a power of two and a factor of 1 to 2: the former is applied together with the
// token's to each wavefront's sum, the latter to the sum of all. So no partial result leaves fp32's range unless the
// scaled one does (x near 1e36: the sum of its products with the codes is beyond), and the roundings are those of sum
// times scale. The lanes that finish do it, with the powers of two through LDS: read earlier, the scales cost registers
// in the loop (int8, 6144 x 6144, 1 token: 12.7 to 13.0 us, 12.3 so).
__device__ __forceinline__ int scale_exp(float s) { return __builtin_amdgcn_frexp_expf(s) - 1; }
__device__ __forceinline__ float scale_factor(float s) { return 2.0f * __builtin_amdgcn_frexp_mantf(s); }

template <class TX, int TOK, int W, int GSH, int F, bool TURNS>
__global__ __launch_bounds__(64 * kTinyWaves, 4) void k_linear_tiny(LinearArgs a) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1;
  constexpr int kRing = W == 8 || F == 2 ? 3 : 4;  // quads of codes in flight
  extern __shared__ __align__(16) _Float16 xs[];   // per wavefront [NX][its blocks][4][TOK][8]
  __shared__ float s_sum[TURNS ? 2 : 1][kTinyWaves][F][TOK][16];
  __shared__ int s_sh[TURNS ? 2 : 1][kTinyWaves][TOK];  // read with one scale a row
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, rt = min(lane & 15, TOK - 1);
  const int nq = (a.nb + 3) / 4, per = (nq + kTinyWaves - 1) / kTinyWaves;
  const int qa = min(wave * per, nq), qb = min(qa + per, nq);
  const int ng = (min(4 * qb, a.nb) - min(4 * qa, a.nb)) * 4;  // granules of a token in the wavefront's columns
  const int tk = lane % TOK, g0 = lane / TOK;
  constexpr int kPer = 64 / TOK, kRounds = tiny_rounds(sizeof(TX));
  Granule<TX> raw[kRounds];
  const TX* xrow = static_cast<const TX*>(a.x) + (size_t)min(tk, a.T - 1) * a.ldx + (size_t)qa * 128;
#pragma unroll
  for (int k = 0; k < kRounds; ++k)
    if (g0 + k * kPer < ng) load8(xrow + (g0 + k * kPer) * 8, a.vec_x, raw[k]);
  __builtin_amdgcn_sched_barrier(0);
  const int outs = a.half ? a.half : a.N;
  constexpr int kOuts = 16;  // of a workgroup at a time
  int out0 = blockIdx.x * kOuts;
  Rows<W, GSH, F> rows(a, out0, lane);
  Quad<W, GSH> ring[kRing][F];
  float scale[F];
  auto begin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < F; ++f) scale[f] = TURNS && GSH < 0 ? *rows.scale[f] : 1.0f;
#pragma unroll
    for (int k = 0; k < kRing; ++k)
      if (qa + k < qb) rows.load(ring[k], 4 * (qa + k));
  };
  begin();
  __builtin_amdgcn_sched_barrier(0);
  bool finite = true;
  int sh = 0;
  if constexpr (!std::is_same<TX, _Float16>::value) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
      if (g0 + k * kPer < ng) amax8<TX>(raw[k], m);
    m = amax_bits<TX>(m);
#pragma unroll
    for (int o = TOK; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    finite = m < 0x7F800000u;
    sh = scale_shift(m);
  }
  _Float16* x = xs + (size_t)wave * NX * per * 128 * TOK;
  const int stride = per * 128 * TOK;
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int gr = g0 + k * kPer;
    if (gr < (qb - qa) * 16) {
      h8 hi = {}, lo = {};
      if (gr < ng) convert8<TX>(raw[k], sh, finite, hi, lo);
      *reinterpret_cast<h8*>(x + (gr * TOK + tk) * 8) = hi;
      if (NX == 2) *reinterpret_cast<h8*>(x + stride + (gr * TOK + tk) * 8) = lo;
    }
  }
  wave_sync();
  f4v acc[1][F];
  auto multiply = [&](Quad<W, GSH> (&d)[F], int q) __attribute__((always_inline)) {
    multiply_quad<NX, 1, TOK, W, GSH, F>(d, x + (q - qa) * 128 * TOK, stride, rt, g, acc);
  };
  for (int buf = 0;; buf ^= TURNS) {
#pragma unroll
    for (int f = 0; f < F; ++f) acc[0][f] = f4v{0.0f, 0.0f, 0.0f, 0.0f};
    int q0 = qa;
    for (; q0 + kRing < qb; q0 += kRing) {
#pragma unroll
      for (int k = 0; k < kRing; ++k) {
        multiply(ring[k], q0 + k);
        rows.load(ring[k], 4 * min(q0 + k + kRing, qb - 1));
      }
    }
#pragma unroll
    for (int k = 0; k < kRing; ++k)
      if (q0 + k < qb) multiply(ring[k], q0 + k);
    // lane group 0 holds the real tokens: row r, token j; token j's power of two is in lane j
    if constexpr (GSH < 0) {
      if (g == 0)
#pragma unroll
        for (int j = 0; j < TOK; ++j)
#pragma unroll
          for (int f = 0; f < F; ++f) s_sum[buf][wave][f][j][lane] = acc[0][f][j];
      if (lane < TOK) s_sh[buf][wave][lane] = sh;
    } else {
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        const int back = -__builtin_amdgcn_readlane(sh, j);
        if (g == 0)
#pragma unroll
          for (int f = 0; f < F; ++f) s_sum[buf][wave][f][j][lane] = ldexpf(acc[0][f][j], back);
      }
    }
    const int at = out0;
    float rs[F];
#pragma unroll
    for (int f = 0; f < F; ++f) rs[f] = scale[f];
    out0 += gridDim.x * kOuts;
    const bool more = TURNS && out0 < outs;
    if (more) {  // the next rows' codes are on their way while these are finished
      rows = Rows<W, GSH, F>(a, out0, lane);
      begin();
    }
    __syncthreads();  // the only one a turn: a buffer is written again two turns on
    const int j = threadIdx.x >> 4, r = threadIdx.x & 15;
    if (threadIdx.x < 16 * TOK && j < a.T) {
      float v[F];
#pragma unroll
      for (int f = 0; f < F; ++f) {
        if constexpr (GSH < 0) {
          const float sc = TURNS ? rs[f] : a.scales[a.half ? f * a.half + at + r : at + r];
          const int e = scale_exp(sc);
          v[f] = ldexpf(s_sum[buf][0][f][j][r], e - s_sh[buf][0][j]);
#pragma unroll
          for (int w = 1; w < kTinyWaves; ++w) v[f] += ldexpf(s_sum[buf][w][f][j][r], e - s_sh[buf][w][j]);
          v[f] *= scale_factor(sc);
        } else {
          v[f] = s_sum[buf][0][f][j][r];
#pragma unroll
          for (int w = 1; w < kTinyWaves; ++w) v[f] += s_sum[buf][w][f][j][r];  // columns in ascending order
        }
      }
      if (a.half) {
        finish<TX>(a, j, at + r, v[0], v[F - 1]);
      } else {
        finish<TX>(a, j, at + r, v[0], 0.0f);
      }
    }
    if (!more) break;
  }
}

// More: a workgroup takes 128 rows (64 gate and 64 up) by 16*NT tokens over a part of the columns, because every
// workgroup reads and converts the activations of its columns; four wavefronts of 32 rows for each half of them. Parts
// are added by k_linear_join. 32 tokens, 4096 x 6144 int4 g64 with SwiGLU: 11.1 us and 2.5 to 3.9 to add, on 15 MB;
// latency: the conversion, then three quads of codes a wavefront, then the sum. A head, 65536 x 6144 int4: 55.8 us for 8
// tokens, 96.6 for 32, on 205 MB: its columns are cut by what the lanes convert, into 3 and 6 parts whose sums are written
// and read.
constexpr int kSlimRowWaves = 4, kSlimColWaves = 2, kSlimLanes = 64 * kSlimRowWaves * kSlimColWaves;
constexpr int kSlimRounds = 8;  // granules that a lane converts, over all token fragments

template <class TX, int NT, int W, int GSH>
__global__ __launch_bounds__(kSlimLanes, 2) void k_linear_slim(LinearArgs a, int kblocks, float* __restrict__ part) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1, F = 2, RW = kSlimRowWaves;
  constexpr int kPer = kSlimLanes / 16, kRounds = kSlimRounds / NT, kRing = 3;
  extern __shared__ __align__(16) _Float16 xs[];  // [NX][NT][nq * 4 blocks][4][16][8]; later the second half's sums
  __shared__ uint32_t s_max[kSlimLanes / 64][NT * 16];
  __shared__ int s_sh[NT * 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int rw = wave % RW, kw = wave / RW;
  const int b0 = blockIdx.y * kblocks, nblk = min(kblocks, a.nb - b0), nq = (nblk + 3) / 4;
  const int t0 = blockIdx.z * 16 * NT;
  const int tk = threadIdx.x & 15, g0 = threadIdx.x >> 4, ng = nblk * 4;
  Granule<TX> raw[NT][kRounds];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const TX* row = static_cast<const TX*>(a.x) + (size_t)min(t0 + 16 * n + tk, a.T - 1) * a.ldx + (size_t)b0 * 32;
#pragma unroll
    for (int k = 0; k < kRounds; ++k)
      if (g0 + k * kPer < ng) load8(row + (g0 + k * kPer) * 8, a.vec_x, raw[n][k]);
  }
  __builtin_amdgcn_sched_barrier(0);
  const int out0 = (blockIdx.x * RW + rw) * (a.half ? 16 : 32);
  const bool any = out0 < (a.half ? a.half : a.N);
  const Rows<W, GSH, F> rows(a, out0, lane);
  const int per = (nq + kSlimColWaves - 1) / kSlimColWaves;
  const int qa = min(kw * per, nq), qb = min(qa + per, nq);  // this wavefront's quads
  Quad<W, GSH> ring[kRing][F];
#pragma unroll
  for (int k = 0; k < kRing; ++k)
    if (qa + k < qb) rows.load(ring[k], b0 + 4 * (qa + k));
  __builtin_amdgcn_sched_barrier(0);

  bool finite[NT];
  int sh[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) finite[n] = true, sh[n] = 0;
  if constexpr (!std::is_same<TX, _Float16>::value) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kRounds; ++k)
        if (g0 + k * kPer < ng) amax8<TX>(raw[n][k], m);
      m = amax_bits<TX>(m);
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lane < 16) s_max[wave][n * 16 + tk] = m;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kSlimLanes / 64; ++w) m = max(m, s_max[w][n * 16 + tk]);
      finite[n] = m < 0x7F800000u;
      sh[n] = scale_shift(m);
    }
  }
  if (g0 == 0)
#pragma unroll
    for (int n = 0; n < NT; ++n) s_sh[n * 16 + tk] = sh[n];
  const int stride = nq * 2048;  // halfs of a token fragment
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
      const int gr = g0 + k * kPer;
      if (gr < nq * 16) {
        h8 hi = {}, lo = {};
        if (gr < ng) convert8<TX>(raw[n][k], sh[n], finite[n], hi, lo);
        *reinterpret_cast<h8*>(xs + n * stride + (gr * 16 + tk) * 8) = hi;
        if (NX == 2) *reinterpret_cast<h8*>(xs + (NT + n) * stride + (gr * 16 + tk) * 8) = lo;
      }
    }
  __syncthreads();

  f4v acc[NT][F];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[n][f] = f4v{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](Quad<W, GSH> (&d)[F], int q) __attribute__((always_inline)) {
    multiply_quad<NX, NT, 16, W, GSH, F>(d, xs + q * 2048, stride, r, g, acc);
  };
  int q0 = qa;
  for (; q0 + kRing < qb; q0 += kRing) {
#pragma unroll
    for (int k = 0; k < kRing; ++k) {
      multiply(ring[k], q0 + k);
      rows.load(ring[k], b0 + 4 * min(q0 + k + kRing, qb - 1));
    }
  }
#pragma unroll
  for (int k = 0; k < kRing; ++k)
    if (q0 + k < qb) multiply(ring[k], q0 + k);

  // first half of the columns plus second
  f4v* sums = reinterpret_cast<f4v*>(xs);  // [RW][NT][F][64 lanes]
  __syncthreads();
  if (kw > 0) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int f = 0; f < F; ++f) sums[((rw * NT + n) * F + f) * 64 + lane] = acc[n][f];
  }
  __syncthreads();
  if (kw > 0 || !any) return;
  float rs[F];
#pragma unroll
  for (int f = 0; f < F; ++f) rs[f] = GSH < 0 ? *rows.scale[f] : 1.0f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int f = 0; f < F; ++f) acc[n][f] += sums[((rw * NT + n) * F + f) * 64 + lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tt = 16 * n + 4 * g + j, t = t0 + tt;
      if (t >= a.T) continue;
      const int back = -s_sh[tt];
      float v[F];
#pragma unroll
      for (int f = 0; f < F; ++f) v[f] = ldexpf(acc[n][f][j] * rs[f], back);
      if (part) {
#pragma unroll
        for (int f = 0; f < F; ++f) part[((size_t)blockIdx.y * a.T + t) * a.N + rows.row[f]] = v[f];
      } else if (a.half) {
        finish<TX>(a, t, rows.row[0], v[0], v[1]);
      } else {
#pragma unroll
        for (int f = 0; f < F; ++f) finish<TX>(a, t, rows.row[f], v[f], 0.0f);
      }
    }
  }
}

// Adds the parts in ascending order and finishes; one output a lane, kJoinLoads parts read at once.
constexpr int kJoinLoads = 16;
template <class TX>
__global__ __launch_bounds__(256) void k_linear_join(LinearArgs a, const float* __restrict__ part, int parts) {
  const int out = a.half ? a.half : a.N;
  const int col = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (col >= out) return;
  const size_t step = (size_t)a.T * a.N;
  const float* p = part + (size_t)t * a.N + col;
  float v = 0.0f, u = 0.0f;
  for (int k0 = 0; k0 < parts; k0 += kJoinLoads) {
    float b[kJoinLoads], c[kJoinLoads];
#pragma unroll
    for (int k = 0; k < kJoinLoads; ++k) {
      const size_t at = (size_t)min(k0 + k, parts - 1) * step;
      b[k] = p[at];
      if (a.half) c[k] = p[at + a.half];
    }
#pragma unroll
    for (int k = 0; k < kJoinLoads; ++k)
      if (k0 + k < parts) {
        v += b[k];
        if (a.half) u += c[k];
      }
  }
  finish<TX>(a, t, col, v, u);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Where the codes' way through memory, and having enough workgroups, counts more than the products: up to 32 tokens, and
// up to kSlimWork tokens times rows, at which the tiles below take as long (64 tokens x 6144 rows: 16 us over 2048
// columns either way, 32 and 29 over 6144; 192 x 2048: 16 either way, 30 and 30; 32 tokens x 65536 rows over 6144: 97
// here, 33 tokens in tiles 97).
constexpr int kSlimTokens = 32;
constexpr int64_t kSlimWork = 3 << 17;
constexpr int kTinyTokens = 4;
constexpr int kSlimGroups = 256;  // workgroups wanted: one per compute unit
bool is_slim(int64_t T, int N) { return T <= kSlimTokens || T * N <= kSlimWork; }

// up to 4 tokens whose columns fit the lanes' rounds, and the activations 64 KB; size: bytes of an activation
bool tiny_fits(int64_t T, int K, int size) {
  const int tok = T == 1 ? 1 : kTinyTokens, quads = (K / 32 + 3) / 4, per = (quads + kTinyWaves - 1) / kTinyWaves;
  return T <= kTinyTokens && per * 16 * tok <= tiny_rounds(size) * 64 &&
         kTinyWaves * per * 256 * tok * (size == 4 ? 2 : 1) <= 64 << 10;
}
int slim_frags(int64_t T) { return T <= 16 ? 1 : 2; }

// Columns are cut so that about kSlimGroups workgroups run, in parts of whole quads of blocks that the lanes' rounds
// cover.
struct SlimPlan {
  int kblocks, parts;
};
SlimPlan slim_plan(int N, int nb, int nt, int64_t T) {
  const int groups = (N + 127) / 128 * (int)((T + 16 * nt - 1) / (16 * nt)), quads = (nb + 3) / 4;
  const int most = kSlimRounds / nt * (kSlimLanes / 16) / 16;
  int parts = std::max(1, std::min(quads, kSlimGroups / groups));
  const int per = std::min((quads + parts - 1) / parts, most);
  parts = (quads + per - 1) / per;
  return {per * 4, parts};
}

struct LinearPlan {
  size_t xh, xl, sh, total;
};
LinearPlan linear_plan(int K, int64_t T) {
  LinearPlan p;
  const size_t nbp = (size_t)((K / 32 + 1) & ~1), tp = (size_t)((T + 31) / 32) * 32;
  const size_t x = up256(tp * nbp * 32 * 2);
  p.xh = 0;
  p.xl = x;
  p.sh = 2 * x;
  p.total = p.sh + up256((size_t)T * 4);
  return p;
}
size_t slim_bytes(int N, int K, int64_t T) {
  const SlimPlan s = slim_plan(N, K / 32, slim_frags(T), T);
  return s.parts > 1 ? (size_t)s.parts * T * N * 4 : 0;
}

template <class TX, int TOK, int F, int W, int GSH>
void tiny_launch(const LinearArgs& a, hipStream_t st) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1;
  const int quads = (a.nb + 3) / 4, per = (quads + kTinyWaves - 1) / kTinyWaves;
  const int rows = (a.half ? a.half : a.N) / 16, turns = (rows + kTinyGroups - 1) / kTinyGroups;
  const size_t lds = (size_t)kTinyWaves * per * 256 * TOK * NX;
  if (F == 1 && turns > 3)
    k_linear_tiny<TX, TOK, W, GSH, F, F == 1><<<(rows + turns - 1) / turns, 64 * kTinyWaves, lds, st>>>(a);
  else
    k_linear_tiny<TX, TOK, W, GSH, F, false><<<rows, 64 * kTinyWaves, lds, st>>>(a);
}
template <class TX, int NT, int W, int GSH>
void slim_launch(const LinearArgs& a, float* ws, hipStream_t st) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1;
  const SlimPlan s = slim_plan(a.N, a.nb, NT, a.T);
  const int nq = std::min(s.kblocks / 4, (a.nb + 3) / 4);
  const size_t lds = std::max((size_t)NX * NT * nq * 4096, (size_t)kSlimRowWaves * NT * 2 * 64 * 16);
  const int out = a.half ? a.half : a.N, per = a.half ? 64 : 128;
  float* part = s.parts > 1 ? ws : nullptr;
  k_linear_slim<TX, NT, W, GSH><<<dim3((out + per - 1) / per, s.parts, (a.T + 16 * NT - 1) / (16 * NT)), kSlimLanes, lds, st>>>(a, s.kblocks, part);
  if (part) k_linear_join<TX><<<dim3((out + 255) / 256, a.T), 256, 0, st>>>(a, part, s.parts);
}
template <class TX, int W, int GSH>
void few_tokens(const LinearArgs& a, float* ws, hipStream_t st) {
  if (tiny_fits(a.T, a.K, sizeof(TX))) {
    if (a.T == 1) {
      if (a.half) tiny_launch<TX, 1, 2, W, GSH>(a, st);
      else tiny_launch<TX, 1, 1, W, GSH>(a, st);
    } else {
      if (a.half) tiny_launch<TX, kTinyTokens, 2, W, GSH>(a, st);
      else tiny_launch<TX, kTinyTokens, 1, W, GSH>(a, st);
    }
  } else if (a.T <= 16) {
    slim_launch<TX, 1, W, GSH>(a, ws, st);
  } else {
    slim_launch<TX, 2, W, GSH>(a, ws, st);
  }
}

// More tokens. What fills the card twice over (two workgroups on each of 256 compute units) runs in whole tiles of four
// wavefronts; of what is left, up to 256 tiles run one a compute unit, with eight wavefronts that share the columns, and
// fewer than that are cut into halves or quarters first. Each step against the one before it, us: 128 x 256 tiles, 256
// of them 103 against 111, 128 44.7 / 62.6, 48 22.0 / 28.1 (2,048 columns; 6,144 42.4 / 71.8), 24 22.0 / 30.6; 64 x 256
// tiles of group scales 384 of them 88 / 87, 192 52.7 / 63.9, 96 39.1 / 50.9, 48 25.6 / 38.5, of fp32 111 / 119, 77 / 75,
// 42 / 74, 30 / 40.
constexpr int kUnits = 256;
template <class TX, int W, int GSH>
void tile_launch(const LinearArgs& a, hipStream_t st) {
  constexpr int BT = base_frags<TX, GSH>(), KQ = GSH >= 0 ? 2 : 4;
  const int row_tiles = (a.N + 255) / 256, tok_tiles = (a.T + 32 * BT - 1) / (32 * BT);
  const int tiles = row_tiles * tok_tiles;
  for (int at = 0, left; (left = tiles - at) > 0;) {
    if constexpr (BT == 4) {
      if (left >= 2 * kUnits) {
        const int n = left / (2 * kUnits) * (2 * kUnits);
        k_linear_tile<TX, 4, W, GSH, 4, 1><<<n, 256, 0, st>>>(a, row_tiles, tok_tiles, at, n);
        at += n;
      } else if (left > kUnits / 2) {
        const int n = std::min(left, kUnits);
        k_linear_tile<TX, 4, W, GSH, 4, 2><<<n, 512, 0, st>>>(a, row_tiles, tok_tiles, at, n);
        at += n;
      } else if (left > kUnits / 4) {
        k_linear_tile<TX, 2, W, GSH, 4, 2><<<2 * left, 512, 0, st>>>(a, row_tiles, tok_tiles, at, left);
        at += left;
      } else if (left > kUnits / 8) {
        k_linear_tile<TX, 1, W, GSH, 4, 4><<<4 * left, 1024, 0, st>>>(a, row_tiles, tok_tiles, at, left);
        at += left;
      } else {
        k_linear_tile<TX, 1, W, GSH, 2, 8><<<8 * left, 1024, 0, st>>>(a, row_tiles, tok_tiles, at, left);
        at += left;
      }
    } else {
      // fp32 with a scale a block: 64 tokens take too many registers (2,048 tokens 12288 x 4096: 466 us with 32, 488)
      constexpr bool kWhole = GSH != 0 || !std::is_same<TX, float>::value;
      int n = left;
      if (kWhole && left >= 2 * kUnits) {
        // a last turn of few tiles is cut too (bf16 with group scales, us: 64 over 134 whole, 114 cut; 32 118 / 109; fp32 128
        // 281 / 282; 176 210 / 216; 400 190 / 220)
        const int over = left % (2 * kUnits);
        n = over > kUnits / 2 ? left : left - over;
        k_linear_tile<TX, kWhole ? 2 : 1, W, GSH, 4, 1><<<n, 256, 0, st>>>(a, row_tiles, tok_tiles, at, n);
      } else if (left > kUnits) {
        k_linear_tile<TX, 1, W, GSH, 4, 1><<<2 * left, 256, 0, st>>>(a, row_tiles, tok_tiles, at, left);
      } else if (left > kUnits / 2) {
        k_linear_tile<TX, 2, W, GSH, 4, 2><<<left, 512, 0, st>>>(a, row_tiles, tok_tiles, at, left);
      } else if (left > kUnits / 4) {
        k_linear_tile<TX, 1, W, GSH, 4, KQ><<<2 * left, 256 * KQ, 0, st>>>(a, row_tiles, tok_tiles, at, left);
      } else {
        k_linear_tile<TX, 1, W, GSH, 2, 2 * KQ><<<4 * left, 256 * KQ, 0, st>>>(a, row_tiles, tok_tiles, at, left);
      }
      at += n;
    }
  }
}

template <class TX>
void linear_launch(const LinearArgs& a, int bits, void* ws, hipStream_t st) {
  if (is_slim(a.T, a.N)) {
    float* p = static_cast<float*>(ws);
    if (bits == 8) few_tokens<TX, 8, -1>(a, p, st);
    else if (a.gshift < 0) few_tokens<TX, 4, -1>(a, p, st);
    else if (a.gshift == 0) few_tokens<TX, 4, 0>(a, p, st);
    else if (a.gshift == 1) few_tokens<TX, 4, 1>(a, p, st);
    else few_tokens<TX, 4, 2>(a, p, st);
    return;
  }
  k_linear_x<TX><<<(a.T + 31) / 32 * 4, 8 * kPrepLanes, 0, st>>>(a);
  if (bits == 8) tile_launch<TX, 8, -1>(a, st);
  else if (a.gshift < 0) tile_launch<TX, 4, -1>(a, st);
  else if (a.gshift == 0) tile_launch<TX, 4, 0>(a, st);
  else tile_launch<TX, 4, 1>(a, st);
}

}  // namespace

// for any number of tokens up to T
size_t linear_ws_bytes(const moe_linear_config& c, int64_t T) {
  size_t b = is_slim(T, c.rows) ? 256 : linear_plan(c.cols, T).total;
  const int64_t most = std::min(T, std::max<int64_t>(kSlimTokens, kSlimWork / c.rows));
  b = std::max(b, slim_bytes(c.rows, c.cols, std::min<int64_t>(T, 16)));
  for (int64_t t = 32; t < most + 32; t += 32) b = std::max(b, slim_bytes(c.rows, c.cols, std::min(t, most)));
  return b;
}

hipError_t launch_linear(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                         const void* x, int64_t ldx, int T, int dtype, const void* res, int64_t ldr, void* y,
                         int64_t ldy, void* ws, hipStream_t st) {
  LinearArgs a{};
  a.T = T;
  a.N = c.rows;
  a.K = c.cols;
  a.nb = c.cols / 32;
  a.nbp = (a.nb + 1) & ~1;
  a.half = c.act == MOE_ACT_SWIGLU ? c.rows / 2 : 0;
  a.act = c.act;
  const size_t elem = dtype == MOE_DTYPE_F32 ? 4 : 2;
  a.vec_x = aligned16(x) && (size_t)ldx * elem % 16 == 0;
  a.vec_r = reinterpret_cast<uintptr_t>(res) % (4 * elem) == 0 && ldr % 4 == 0;
  a.vec_y = reinterpret_cast<uintptr_t>(y) % (4 * elem) == 0 && ldy % 4 == 0;
  a.gshift = -1;
  if (c.group_size > 0)
    for (a.gshift = 0; (32 << a.gshift) < c.group_size;) ++a.gshift;
  a.codes = codes;
  a.scales = scales;
  a.bias = bias;
  a.x = x;
  a.res = res;
  a.y = y;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  const LinearPlan p = linear_plan(c.cols, T);
  char* w = static_cast<char*>(ws);
  a.xh = reinterpret_cast<_Float16*>(w + p.xh);
  a.xl = reinterpret_cast<_Float16*>(w + p.xl);
  a.sh = reinterpret_cast<int32_t*>(w + p.sh);
  const int bits = c.weight_bits == 8 ? 8 : 4;
  if (dtype == MOE_DTYPE_F32) linear_launch<float>(a, bits, ws, st);
  else if (dtype == MOE_DTYPE_BF16) linear_launch<bf16_t>(a, bits, ws, st);
  else linear_launch<_Float16>(a, bits, ws, st);
  return hipGetLastError();
}

}  // namespace moe
