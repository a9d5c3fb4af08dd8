// k_linear.hip — y = act(W x + b) + r over the library's row-tiled int4 / int8 codes, activations in fp32, bf16 or
// fp16 and not quantized.
//
// Both operands go to the matrix cores as fp16, without loss:
//  - a code (at most 8 bits) is an integer that fp16 holds exactly; its scale multiplies the fp32 sum.
//  - an activation is multiplied by a power of two per token, such that the token's largest lies in [2^14, 2^15).
//    fp16 then holds every bf16 value down to 2^-32 of the largest exactly, and any smaller one to 2^-39 of the
//    largest. fp32 values are split, v = hi + lo, both fp16: what is lost is below 2^-23 of the value (or 2^-39 of
//    the token's largest). fp16 values are taken as they are.
// Products are exact in fp32, sums are fp32.
//
// Unpacking a word of eight nibbles: the nibble, moved to 0..15 by flipping its top bit, is put into the low (or
// next) mantissa bits of 1024.0; a packed subtraction (or multiply-add by 1/16) leaves the code. That gives the
// element order 0 4 1 5 2 6 3 7, in which the activations are stored too.
#include <type_traits>

#include "moe_float.h"
#include "moe_internal.h"

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

// ------------------------------------------------------------ activations to fp16 in tile order
// One workgroup takes 8 tokens: thread = (token tid % 8, granule of 8 elements tid / 8), so 8 neighbouring threads
// write 128 contiguous bytes and each token is read in runs of 32 granules.
template <class TX>
__global__ __launch_bounds__(256) void k_linear_x(LinearArgs a) {
  __shared__ uint32_t s_max[32][8];
  const int tk = threadIdx.x & 7, g0 = threadIdx.x >> 3;
  const int t = blockIdx.x * 8 + tk;
  const bool in = t < a.T;
  const TX* row = static_cast<const TX*>(a.x) + (size_t)(in ? t : 0) * a.ldx;
  const int ng = a.K / 8;
  constexpr bool kScaled = !std::is_same<TX, _Float16>::value;
  int sh = 0;
  bool finite = true;
  if (kScaled) {
    uint32_t m = 0;
    if (in)
      for (int g = g0; g < ng; g += 32)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(to_f32<TX>(row[g * 8 + i])) & 0x7FFFFFFFu);
    s_max[g0][tk] = m;
    __syncthreads();
    for (int i = 0; i < 32; ++i) m = max(m, s_max[i][tk]);
    finite = m < 0x7F800000u;
    sh = finite && m > 0 ? 14 - ((int)(m >> 23) - 127) : 0;
  }
  if (in && g0 == 0) a.sh[t] = sh;
  const size_t base = (size_t)(t >> 5) * a.nbp * 1024 + (size_t)(t & 31) * 8;
  for (int g = g0; g < a.nbp * 4; g += 32) {
    h8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = (i >> 1) + 4 * (i & 1);  // element order 0 4 1 5 2 6 3 7
      float v = in && g < ng ? to_f32<TX>(row[g * 8 + e]) : 0.0f;
      if (kScaled) {
        v = ldexpf(v, sh);
        if (!finite && fabsf(v) < INFINITY) v = fminf(fmaxf(v, -65504.0f), 65504.0f);
      }
      hi[i] = (_Float16)v;
      lo[i] = (_Float16)(fabsf(v) < INFINITY ? v - (float)hi[i] : 0.0f);
    }
    const size_t at = base + (size_t)g * 256;  // g = block * 4 + slice
    *reinterpret_cast<h8*>(a.xh + at) = hi;
    if (std::is_same<TX, float>::value) *reinterpret_cast<h8*>(a.xl + at) = lo;
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
    case MOE_ACT_RELU: return v > 0.0f ? v : 0.0f;
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

// ------------------------------------------------------------ product
// A wavefront multiplies 32*TT tokens by two fragments of 32 weight rows (64 consecutive rows; with SwiGLU 32 gate
// rows and the 32 up rows that go with them) with v_mfma_f32_32x32x16_f16. Four wavefronts of a workgroup share the
// tokens, whose activations pass through LDS; each reads its own codes from memory into registers.
// Lane l: token / weight row l % 32, half g = l / 32 of a block. Result: weight row l % 32, tokens
// 8*(i/4) + 4*g + i%4.
template <class TX, int TT, int W, bool GS>
__global__ __launch_bounds__(256) void k_linear_tile(LinearArgs a) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1;
  constexpr int kStep = TT * NX * 2 * 1024;  // halfs of a block pair: [NX][TT][2 blocks][4 slices][32][8]
  __shared__ __align__(16) _Float16 s_x[kStep];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, g = lane >> 5;
  const int cols = a.half ? a.half / 32 : a.N / 64;  // wavefront tiles over the outputs
  const int wt = blockIdx.x * 4 + wave;
  const int t0 = blockIdx.y * 32 * TT;
  const int wtc = min(wt, cols - 1);
  int row[2];
  row[0] = a.half ? wtc * 32 + r : wtc * 64 + r;
  row[1] = a.half ? a.half + wtc * 32 + r : wtc * 64 + 32 + r;
  const uint8_t* src[2];
#pragma unroll
  for (int f = 0; f < 2; ++f)
    src[f] = a.codes + tbw_off<W>(row[f] / 64, 0, a.nb) + (size_t)(row[f] % 64) * (4 * W);
  f16v acc[TT][2];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[tt][f][i] = 0.0f;
  const int groups = GS ? a.nb >> a.gshift : 0;
  for (int b = 0; b < a.nbp; b += 2) {
    __syncthreads();
    for (int i = threadIdx.x; i < kStep / 8; i += 256) {
      const int n = i / (TT * 256), tt = i / 256 % TT, rest = i % 256;
      const int tg = min(t0 / 32 + tt, (a.T - 1) / 32);
      const _Float16* p = (n ? a.xl : a.xh) + ((size_t)tg * a.nbp + b) * 1024 + (size_t)rest * 8;
      *reinterpret_cast<h8*>(s_x + (size_t)i * 8) = *reinterpret_cast<const h8*>(p);
    }
    __syncthreads();
    u4v w[2][W / 4];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const u4v* p = reinterpret_cast<const u4v*>(src[f] + (size_t)min(b + g, a.nb - 1) * kTileBlock<W>);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) w[f][i] = p[i];
      // half g of both blocks instead of all of block b + g
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        constexpr int hv = W / 4 - 1, ho = W == 4 ? 2 : 0;
        const auto sw = __builtin_amdgcn_permlane32_swap(w[f][0][i], w[f][hv][i + ho], false, false);
        w[f][0][i] = sw[0];
        w[f][hv][i + ho] = sw[1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // block b + h
      h8 wf[2][2];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          wf[f][m] = W == 4 ? codes_h8(w[f][0][2 * h + m]) : codes_h8(w[f][h & (W / 4 - 1)][2 * m], w[f][h & (W / 4 - 1)][2 * m + 1]);
      float sc[2];
      if (GS) {
        const int gi = min(b + h, a.nb - 1) >> a.gshift;
#pragma unroll
        for (int f = 0; f < 2; ++f) sc[f] = a.scales[((size_t)(row[f] / 64) * groups + gi) * 64 + row[f] % 64];
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          f16v c;
          if (GS) {
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i] = 0.0f;
          } else {
            c = acc[tt][f];
          }
#pragma unroll
          for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const h8 xf = *reinterpret_cast<const h8*>(
                  s_x + ((size_t)((n * TT + tt) * 2 + h) * 4 + 2 * g + m) * 256 + r * 8);
              c = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, wf[f][m], c, 0, 0, 0);
            }
          if (GS) {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[tt][f][i] = fmaf(c[i], sc[f], acc[tt][f][i]);
          } else {
            acc[tt][f] = c;
          }
        }
    }
  }
  if (wt >= cols) return;
  float rs[2] = {1.0f, 1.0f};
  if (!GS) {
    rs[0] = a.scales[row[0]];
    rs[1] = a.scales[row[1]];
  }
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = t0 + 32 * tt + 8 * (i >> 2) + 4 * g + (i & 3);
      if (t >= a.T) continue;
      const int sh = -a.sh[t];
      const float v0 = ldexpf(acc[tt][0][i] * rs[0], sh), v1 = ldexpf(acc[tt][1][i] * rs[1], sh);
      if (a.half) {
        finish<TX>(a, t, wt * 32 + r, v0, v1);
      } else {
        finish<TX>(a, t, row[0], v0, 0.0f);
        finish<TX>(a, t, row[1], v1, 0.0f);
      }
    }
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

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

template <class TX>
void linear_launch(const LinearArgs& a, int bits, hipStream_t st) {
  k_linear_x<TX><<<(a.T + 31) / 32 * 4, 256, 0, st>>>(a);
  const int cols = a.half ? a.half / 32 : a.N / 64;
  const dim3 grid((cols + 3) / 4, (a.T + 31) / 32);
  if (bits == 8) k_linear_tile<TX, 1, 8, false><<<grid, 256, 0, st>>>(a);
  else if (a.gshift >= 0) k_linear_tile<TX, 1, 4, true><<<grid, 256, 0, st>>>(a);
  else k_linear_tile<TX, 1, 4, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

size_t linear_ws_bytes(const moe_linear_config& c, int64_t T) { return linear_plan(c.cols, T).total; }

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
  if (dtype == MOE_DTYPE_F32) linear_launch<float>(a, bits, st);
  else if (dtype == MOE_DTYPE_BF16) linear_launch<bf16_t>(a, bits, st);
  else linear_launch<_Float16>(a, bits, st);
  return hipGetLastError();
}

}  // namespace moe
