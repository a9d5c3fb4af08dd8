// k_linear_grad.hip — gradients of y = act(W x + b + s B (A x)) for frozen codes W: with dz = dy act'(z),
//   dx = W^T dz + s A^T (B^T dz),  dB = sum over tokens of dz (s A x)^T,  dA = sum over tokens of (s B^T dz) x^T.
// W^T dz runs in the product's tiles, summing over the weight rows. Row scales are multiplied into dz, in fp32 before its
// one rounding to fp16 (relative 2^-11; fp32 gradients keep two halves, 2^-23). Two halves for fp16 gradients too would make
// them as exact as their type (2.1e-4 in the 2-norm for 2.9e-4) and take 1.8 times as long: 2,048 tokens 12288 x 6144 SwiGLU
// 327 us, 599 in fp32; bf16's own rounding is 1.7e-3. Group scales differ along a row: the power of two of a row's largest
// is multiplied into dz, without loss, what is left of them, at most 2^12 (times a code of at most 8 it fits fp16), into the
// codes. bf16 gradients take it as one fp16 (two roundings, 2^-10 of a weight). fp16 and fp32 gradients take eight bits of it,
// whose product with a code is exact, and the rest as a second fp16 (its rounding and its product's, 2^-20 and 2^-19); the
// product of that with the second half of an fp32 dz, 2^-19 more, is left out. Below fp16's normal range, for scales less
// than 2^-25 of their row's largest and in two parts 2^-17, both roundings are 2^-25 in place, 2^-36 of that largest each at
// most. For the adapters' sums dz is kept in fp32: rounding it to the call's type makes bf16 d_a and d_b 1.4 times as far off
// (2.3e-3 in the 2-norm for 1.7e-3), and fp16 values beyond 65504 infinite (2,000 tokens, 4096 rows, SwiGLU, rank 32: dz,
// s (B^T dz) and d_a, d_b take 61 us, 50 with it).
#define MOE_ADAPTED 1
#define MOE_TRANSPOSED 1
#include "linear_kernels.h"

namespace moe {

namespace {

// ------------------------------------------------------------ dz
// Derivative of the activation. Beyond 1e9 it is its limit (and no infinity meets a zero); NaN stays.
__device__ __forceinline__ float slope(float z, int act) {
  float s, miss;
  if (act == MOE_ACT_RELU) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);
  const float v = z != z ? z : fminf(fmaxf(z, -1e9f), 1e9f);
  switch (act) {
    case MOE_ACT_SILU: sigmoid2(v, s, miss); return fmaf(v * s, miss, s);
    case MOE_ACT_GELU: return fmaf(v * 0.398942280f, exp_neg(-0.5f * v * v), 0.5f * erfcf(v * -0.707106781f));
    case MOE_ACT_GELU_TANH:
      sigmoid2(1.59576912f * v * fmaf(0.044715f * v, v, 1.0f), s, miss);
      return fmaf(v * s * miss, 1.59576912f * fmaf(0.134145f * v, v, 1.0f), s);
    default: return 1.0f;
  }
}

struct DzArgs {
  LinearArgs a;      // xh, xl, sh, order, T of the tiles that follow
  const void* dy;
  const void* pre;
  int64_t ldd, ldp;
  int32_t vec_d, vec_p;
  int32_t N, half, act;  // weight rows, those of the gate part, activation
  const float* mul;      // [N] row scales, or the power of two of the group scales; nullptr: no product follows
  float* dz;             // [T][N] by position, or nullptr
};

// dz of eight neighbouring rows n, kind 2 (SwiGLU): of eight gate rows and the up rows that go with them.
template <class TX, int KIND>
__device__ __forceinline__ void dz8(const DzArgs& d, int64_t t, int n, f8v (&o)[KIND == 2 ? 2 : 1]) {
  Granule<TX> g, z, u;
  load8(static_cast<const TX*>(d.dy) + t * d.ldd + n, d.vec_d, g);
  const TX* p = static_cast<const TX*>(d.pre) + t * d.ldp + n;
  if (KIND > 0) load8(p, d.vec_p, z);
  if (KIND == 2) load8(p + d.half, d.vec_p, u);
  const f8v v = granule_f32<TX>(g);
  o[0] = v;
  if constexpr (KIND == 1) {
    const f8v zv = granule_f32<TX>(z);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[0][i] = v[i] * slope(zv[i], d.act);
  }
  if constexpr (KIND == 2) {
    const f8v zv = granule_f32<TX>(z), uv = granule_f32<TX>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // gate beyond 1e9: the limits of silu and of its derivative, so that no infinity meets a zero
      const float c = zv[i] != zv[i] ? zv[i] : fminf(fmaxf(zv[i], -1e9f), 1e9f);
      float s, miss;
      sigmoid2(c, s, miss);
      // dy up may be beyond fp32 where a closed gate leaves little of it; then dy is above 1, and dy silu'(gate) in range
      const float d = fmaf(c * s, miss, s), both = v[i] * uv[i];
      o[0][i] = fabsf(both) < INFINITY ? both * d : v[i] * d * uv[i];
      o[1][i] = v[i] * (zv[i] < -1e9f ? 0.0f : zv[i] * s);
    }
  }
}

// Eight values between the search for a token's largest and the conversion: fp32 as they are, for 16-bit types already as
// fp16 over a power of two of their own, which takes half the registers and is the only rounding (but for values far
// below the token's largest).
template <class TX>
struct Held {
  h8 v;
  int sh;
};
template <>
struct Held<float> {
  f8v v;
};
template <class TX>
__device__ __forceinline__ void hold(const f8v& w, uint32_t& m, Held<TX>& o) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(w[i]) & 0x7FFFFFFFu);
  m = max(m, top);
  if constexpr (std::is_same<TX, float>::value) {
    o.v = w;
  } else {
    o.sh = scale_shift(top);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = ldexpf(w[(i >> 1) + 4 * (i & 1)], o.sh);
      if (top >= 0x7F800000u && fabsf(x) < INFINITY) x = fminf(fmaxf(x, -65504.0f), 65504.0f);
      o.v[i] = (_Float16)x;
    }
  }
}

// As k_linear_x, from dz: TOK positions a workgroup, the largest of a token first. kind: 0 no activation, 1 one row at a
// time, 2 SwiGLU. A row's values stay in registers between the search for the largest and the conversion as far as they fit
// (kRounds items of a lane), the rest is computed twice. One position a workgroup where there are few. 2,048 tokens of 12288
// rows, SwiGLU: 31 to 37 us for 125 MB (20 at the rate of a large read); a workgroup a compute unit, its reading, its
// arithmetic and its writing one after the other. Written one position at a time, in pieces of 16 bytes, it takes 60.
template <class TX, int KIND, int TOK>
__global__ __launch_bounds__(1024) void k_linear_dz(DzArgs d) {
  constexpr int kLanes = 1024 / TOK, V = KIND == 2 ? 2 : 1;
  constexpr int kRounds = TOK == 1 ? 2 : (std::is_same<TX, float>::value ? 8 : 12) / V;
  __shared__ uint32_t s_max[16][TOK];
  const LinearArgs& a = d.a;
  const int tk = threadIdx.x % TOK, g0 = threadIdx.x / TOK;
  const int p = blockIdx.x * TOK + tk;
  const bool in = p < a.T;
  const int64_t t = in ? token_of(a, p) : 0;
  const int items = d.N / V / 8, ng = in ? items : 0;
  Held<TX> v[kRounds][V];
  uint32_t m = 0;
  auto scaled = [&](int g, bool keep, Held<TX> (&o)[V]) __attribute__((always_inline)) {
    f8v w[V];
    dz8<TX, KIND>(d, t, g * 8, w);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int n = k * d.half + g * 8;
      if (keep && d.dz) {
        f4v* to = reinterpret_cast<f4v*>(d.dz + (size_t)p * d.N + n);
        to[0] = f4v{w[k][0], w[k][1], w[k][2], w[k][3]};
        to[1] = f4v{w[k][4], w[k][5], w[k][6], w[k][7]};
      }
      if (d.mul) {
        const f8v s = *reinterpret_cast<const f8v*>(d.mul + n);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[k][i] *= s[i];
        hold<TX>(w[k], m, o[k]);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kRounds; ++k)
    if (g0 + k * kLanes < ng) scaled(g0 + k * kLanes, true, v[k]);
  for (int g = g0 + kRounds * kLanes; g < ng; g += kLanes) {
    Held<TX> o[V];
    scaled(g, true, o);
  }
  if (!d.mul) return;
#pragma unroll
  for (int o = TOK; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  if ((threadIdx.x & 63) < TOK) s_max[threadIdx.x >> 6][tk] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, s_max[i][tk]);
  // at most 2^100, so that the adapters' part, which takes the same power of two, stays in range beside the smallest scales
  const int sh = min(scale_shift(m), 100);
  const bool finite = m < 0x7F800000u;
  if (in && g0 == 0) a.sh[p] = sh;
  const size_t base = (size_t)(p >> 5) * a.nbp * 1024 + (size_t)(p & 31) * 8;
  auto store = [&](int g, const Held<TX> (&o)[V]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      h8 hi = {}, lo = {};
      if (in) {
        if constexpr (std::is_same<TX, float>::value) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x = ldexpf(o[k].v[(i >> 1) + 4 * (i & 1)], sh);
            if (!finite && fabsf(x) < INFINITY) x = fminf(fmaxf(x, -65504.0f), 65504.0f);
            hi[i] = (_Float16)x;
            lo[i] = fabsf(x) < INFINITY ? (_Float16)(x - (float)hi[i]) : (_Float16)0.0f;
          }
        } else {  // a token with an infinity or NaN: its other values only stay finite, whatever they are
          const int by = finite ? sh - o[k].sh : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) hi[i] = __builtin_amdgcn_ldexph(o[k].v[i], by);
        }
      }
      const size_t at = base + ((size_t)k * (d.half / 8) + g) * 256;
      *reinterpret_cast<h8*>(a.xh + at) = hi;
      if (std::is_same<TX, float>::value) *reinterpret_cast<h8*>(a.xl + at) = lo;
    }
  };
#pragma unroll
  for (int k = 0; k < kRounds; ++k)
    if (g0 + k * kLanes < items) store(g0 + k * kLanes, v[k]);
  for (int g = g0 + kRounds * kLanes; g < items; g += kLanes) {
    Held<TX> o[V] = {};
    if (in) scaled(g, false, o);
    store(g, o);
  }
}

template <class TX, int KIND>
void dz_launch(const DzArgs& d, hipStream_t st) {
  const int padded = (d.a.T + 31) / 32 * 32;
  if (d.a.T <= 1024) k_linear_dz<TX, KIND, 1><<<padded, 1024, 0, st>>>(d);
  else k_linear_dz<TX, KIND, 8><<<padded / 8, 1024, 0, st>>>(d);
}

// ------------------------------------------------------------ group scales
// A workgroup takes the 64 rows of a tile: lane l its row l, four groups at a time. scales [tile][group][64].
__global__ __launch_bounds__(256) void k_group_scales(const float* __restrict__ scales, int groups, float* __restrict__ mul,
                                                      _Float16* __restrict__ gs, int64_t gs_low, int low) {
  __shared__ float s_max[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float* s = scales + (size_t)blockIdx.x * groups * 64 + lane;
  float m = 0.0f;
#pragma unroll 4
  for (int g = wave; g < groups; g += 4) m = fmaxf(m, fabsf(s[(size_t)g * 64]));
  s_max[wave][lane] = m;
  __syncthreads();
  m = fmaxf(fmaxf(s_max[0][lane], s_max[1][lane]), fmaxf(s_max[2][lane], s_max[3][lane]));
  // m = f 2^(e + 12), f in [1/2, 1), but 2^e at least fp32's smallest number
  const int e = m > 0.0f && m < INFINITY ? max(__builtin_amdgcn_frexp_expf(m) - 12, -149) : 0;
  // a row of zeros (padding, pruning) adds nothing, so its dz must not count for the token's power of two
  if (wave == 0) mul[blockIdx.x * 64 + lane] = m > 0.0f ? ldexpf(1.0f, e) : 0.0f;
  // place of row l in the order of the codes: eight rows 0 4 1 5 2 6 3 7
  const int r = lane & 7, at = (lane & ~7) + (r < 4 ? 2 * r : 2 * (r - 4) + 1);
  for (int g = wave; g < groups; g += 4) {
    const float v = ldexpf(s[(size_t)g * 64], -e);
    const size_t o = ((size_t)blockIdx.x * groups + g) * 64 + at;
    if (!low) {
      gs[o] = (_Float16)v;
    } else {  // eight bits, whose product with a code is exact, and the rest
      const float hi = to_f32<bf16_t>(from_f32<bf16_t>(v));
      gs[o] = (_Float16)hi;
      gs[gs_low + o] = (_Float16)(v - (float)(_Float16)hi);
    }
  }
}

// ------------------------------------------------------------ few tokens
// Reading the codes is what counts: a wavefront takes 64 columns and a part of the rows for all tokens, with the codes of
// kAhead steps (64 rows) in flight; it waits for no other before the sum of the workgroup's four. The parts' sums
// [part][T][N] are added by k_few_add, with the adapters' part and the residual. 6144 x 6144 int4, bf16: 9.3 us for one
// token, 11.6 for 32, 14.3 for 64 in two fragments, and 4 to add; 19 MB of codes take 3.0 to 4.0.
constexpr int kFewGroups = 512;  // workgroups wanted
constexpr int kFewWaves = 4;
template <class TX, int TT, int W, int GSH>
__global__ __launch_bounds__(256, 2) void k_linear_few(LinearArgs a, int parts, float* __restrict__ sums) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1, GF = GSH < 0 ? 0 : GSH == 0 ? 2 : 1, WP = GF > 0 ? scaled_parts<TX>() : 1;
  constexpr int kAhead = WP == 2 ? 1 : W == 8 || GF > 0 ? 2 : 3;
  // [wavefronts][128 * W] codes, then [wavefronts][32 * TT][64] sums
  __shared__ __align__(16) uint32_t s_mem[kFewWaves * std::max(128 * W, 2048 * TT)];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
  const int col = blockIdx.x * 64;
  uint32_t* s_w = s_mem + wave * 128 * W;
  const int first[2] = {col, min(col + 32, a.N - 32)}, groups = GSH >= 0 ? a.N / 32 >> a.gshift : 0;
  const int64_t steps = a.nbp / 2, k0 = blockIdx.y * kFewWaves + wave;
  const int p0 = (int)(steps * k0 / (parts * kFewWaves)), p1 = (int)(steps * (k0 + 1) / (parts * kFewWaves));
  const size_t step_bytes = (size_t)(a.N / 32) * kTileBlock<W>, low = a.xl - a.xh;
  const uint8_t* src[2];
  const _Float16* gsrc[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    src[f] = a.codes + (size_t)(first[f] / 32) * kTileBlock<W> + (size_t)lane * (4 * W);
    gsrc[f] = GF > 0 ? a.gs + (size_t)(first[f] / 32 >> a.gshift) * 64 + 16 * g : nullptr;
  }
  uint32_t wn[kAhead][2][W];
  h8 gn[kAhead][GF ? GF : 1][WP][2][2];
  auto fetch_w = [&](int p, uint32_t (&w)[2][W], h8 (&gs)[GF ? GF : 1][WP][2][2]) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const u4v v = __builtin_nontemporal_load(reinterpret_cast<const u4v*>(src[f] + (size_t)p * step_bytes) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[f][4 * i + j] = v[j];
      }
#pragma unroll
    for (int f = 0; f < GF; ++f)
#pragma unroll
      for (int v = 0; v < WP; ++v)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            gs[f][v][h][m] = *reinterpret_cast<const h8*>(gsrc[f] + v * a.gs_low + (size_t)p * groups * 64 + h * 32 + m * 8);
  };
  f16v acc[TT][2];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[tt][f][i] = 0.0f;
  auto step = [&](int p, uint32_t (&w)[2][W], h8 (&gs)[GF ? GF : 1][WP][2][2]) __attribute__((always_inline)) {
    h8 xf[NX][TT][2][2], wf[2][2][2 * WP];
#pragma unroll
    for (int n = 0; n < NX; ++n)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            xf[n][tt][h][m] = *reinterpret_cast<const h8*>(a.xh + n * low + (size_t)tt * a.nbp * 1024 + (size_t)p * 2048 +
                                                           (h * 4 + 2 * g + m) * 256 + r * 8);
    unpack_transposed<W, WP, GF>(s_w, w, gs, wf);
    fetch_w(min(p + kAhead, p1 - 1), w, gs);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
          for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              acc[tt][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf[n][tt][h][m], wf[h][m][f], acc[tt][f], 0, 0, 0);
              if constexpr (WP == 2)
                if (n == 0)
                  acc[tt][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf[n][tt][h][m], wf[h][m][2 + f], acc[tt][f], 0, 0, 0);
            }
  };
  if (p0 < p1) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch_w(min(p0 + k, p1 - 1), wn[k], gn[k]);
    for (int p = p0; p < p1; p += kAhead)
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (p + k < p1) step(p + k, wn[k], gn[k]);
  }
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(s_mem);
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) s_sum[((wave * TT + tt) * 32 + 16 * f + i) * 64 + lane] = acc[tt][f][i];
  __syncthreads();
  const int rc = column_at<W>(r);
  for (int k = wave; k < 32 * TT; k += kFewWaves) {  // sum i of fragment f and tokens tt, of all lanes
    const int tt = k >> 5, f = k >> 4 & 1, i = k & 15;
    const int t = 32 * tt + 8 * (i >> 2) + 4 * g + (i & 3);
    float v = s_sum[k * 64 + lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += s_sum[(w * 32 * TT + k) * 64 + lane];
    if (t < a.T && col + 32 * f < a.N) sums[((size_t)blockIdx.y * a.T + t) * a.N + first[f] + rc] = v;
  }
}

// A workgroup takes a token and 1024 columns, a lane four. ab: A of the adapters as it is, [n][R][N].
template <class TX>
__global__ __launch_bounds__(256) void k_few_add(LinearArgs a, int parts, const float* __restrict__ sums) {
  const int t = blockIdx.y, col = blockIdx.x * 1024 + threadIdx.x * 4;
  if (col >= a.N) return;
  const size_t step = (size_t)a.T * a.N;
  const float* p = sums + (size_t)t * a.N + col;
  f4v v = *reinterpret_cast<const f4v*>(p);
#pragma unroll 8
  for (int k = 1; k < parts; ++k) v += *reinterpret_cast<const f4v*>(p + k * step);
  const int sh = a.sh[t], id = a.h ? adapter_of(a, t) : -1;
  float w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = ldexpf(v[i], -sh);
  if (id >= 0) {
    struct alignas(4 * sizeof(TX)) Four {
      TX v[4];
    };
    const TX* b = static_cast<const TX*>(a.ab) + (size_t)id * a.R * a.N + col;
    const float* h = a.h + (size_t)t * a.R;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int r = 0; r < a.R; ++r) {
      const Four q = *reinterpret_cast<const Four*>(b + (size_t)r * a.N);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = fmaf(h[r], to_f32<TX>(q.v[i]), s[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] += s[i];
  }
  finish4<TX>(a, t, col, 0, w, w);
}

// by the columns alone, so that the sums of fewer tokens are no larger
inline int few_parts(int N, int steps) {
  return std::max(1, std::min(kFewGroups / ((N + 63) / 64), steps / (2 * kFewWaves)));
}
inline size_t few_bytes(int N, int steps, int64_t T) {
  return (size_t)few_parts(N, steps) * std::min<int64_t>(T, kAdaptFewTokens) * N * 4;
}
template <class TX, int W, int GSH>
void few_form(const LinearArgs& a, float* sums, hipStream_t st) {
  const int parts = few_parts(a.N, a.nbp / 2);
  const dim3 grid((a.N + 63) / 64, parts);
  if (a.T <= 32) k_linear_few<TX, 1, W, GSH><<<grid, 256, 0, st>>>(a, parts, sums);
  else k_linear_few<TX, 2, W, GSH><<<grid, 256, 0, st>>>(a, parts, sums);
  k_few_add<TX><<<dim3((a.N + 1023) / 1024, a.T), 256, 0, st>>>(a, parts, sums);
}
template <class TX>
void few_launch(const LinearArgs& a, int bits, float* sums, hipStream_t st) {
  if (bits == 8) few_form<TX, 8, -1>(a, sums, st);
  else if (a.gshift < 0) few_form<TX, 4, -1>(a, sums, st);
  else if (a.gshift == 0) few_form<TX, 4, 0>(a, sums, st);
  else few_form<TX, 4, 1>(a, sums, st);
}

// ------------------------------------------------------------ the whole
struct GradPlan {
  LinearPlan z;
  size_t mul, gs, sums, dz, order, ad, offsets, slot0, n_chunks, runs, chunks, h, ht, u, ut, at, bt, part, part_a, total;
};
GradPlan grad_plan(const moe_linear_config& c, const moe_adapters* ad, int64_t T) {
  GradPlan p;
  p.z = linear_plan(c.rows, T);
  size_t at = p.z.total;
  auto take = [&](size_t bytes) {
    const size_t b = at;
    at += up256(bytes);
    return b;
  };
  const size_t groups = c.group_size > 0 ? c.cols / c.group_size : 0;
  p.mul = take(groups ? (size_t)c.rows * 4 : 0);
  p.gs = take(groups * c.rows * 4);
  p.sums = take(std::max(tile_sums_bytes(c.cols, c.rows / 64, T), few_bytes(c.cols, c.rows / 64, T)));
  if (ad) {
    const size_t R = ad->rank, n = ad->n_adapters, N = c.rows, K = c.cols;
    p.dz = take(c.act != MOE_ACT_NONE ? T * N * 4 : 0);
    p.order = take(T * 4);
    p.ad = take(T * 4);
    p.offsets = take((n + 1) * 4);
    p.slot0 = take(n * 4);
    p.n_chunks = take(8);
    p.runs = take(sizeof(AdaptChunk) * (size_t)adapt_max_runs(T, (int)n));
    p.chunks = take(sizeof(AdaptChunk) * (size_t)adapt_max_chunks(T, (int)n));
    p.h = take(T * R * 4);
    p.ht = take((T + 7) / 8 * 8 * R * 4);
    p.u = take(T * R * 4);
    p.ut = take((T + 7) / 8 * 8 * R * 4);
    p.at = take(n * R * K * 4);
    p.bt = take(n * R * N * 4);
    p.part = take((size_t)kAdaptSlots * R * N * 4);
    p.part_a = take((size_t)kAdaptSlots * R * K * 4);
  }
  p.total = at;
  return p;
}

template <class TX>
hipError_t run(const moe_linear_config& c, const uint8_t* codes, const float* scales, const moe_adapters* ad,
               const int32_t* ids, const void* x, int64_t ldx, int T, int dtype, const void* pre, int64_t ldp,
               const void* dy, int64_t ldd, const void* res, int64_t ldr, void* dx, int64_t ldg, void* da, void* db,
               void* ws, hipStream_t st) {
  const GradPlan p = grad_plan(c, ad, T);
  char* w = static_cast<char*>(ws);
  const int N = c.rows, K = c.cols;
  constexpr size_t elem = sizeof(TX);
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(w + at); };
  auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(w + at); };
  auto vec = [&](const void* q, int64_t ld) { return aligned16(q) && (size_t)ld * elem % 16 == 0; };
#define MOE_TRY(call)                          \
  do {                                         \
    const hipError_t e_ = (call);              \
    if (e_ != hipSuccess) return e_;           \
  } while (0)

  LinearArgs a{};
  a.T = T;
  a.N = K;  // outputs
  a.K = N;  // summed over
  a.nb = a.nbp = N / 32;
  a.act = MOE_ACT_NONE;
  a.gshift = group_shift(c);
  a.codes = codes;
  a.res = res;
  a.y = dx;
  a.ldr = ldr;
  a.ldy = ldg;
  a.vec_r = reinterpret_cast<uintptr_t>(res) % (4 * elem) == 0 && ldr % 4 == 0;
  a.vec_y = reinterpret_cast<uintptr_t>(dx) % (4 * elem) == 0 && ldg % 4 == 0;
  a.xh = reinterpret_cast<_Float16*>(w + p.z.xh);
  a.xl = reinterpret_cast<_Float16*>(w + p.z.xl);
  a.sh = i32(p.z.sh);

  AdaptOrder order{};
  const bool few = T <= kAdaptFewTokens;  // positions are tokens
  if (ad) {
    a.ad = ids;
    a.n_ad = ad->n_adapters;
    a.R = ad->rank;
  }
  if (ad && !few) {
    order = AdaptOrder{i32(p.order), i32(p.ad), i32(p.n_chunks) + 1, reinterpret_cast<AdaptChunk*>(w + p.runs),
                       i32(p.offsets), i32(p.slot0), i32(p.n_chunks), reinterpret_cast<AdaptChunk*>(w + p.chunks)};
    MOE_TRY(launch_adapt_order(ids, T, ad->n_adapters, order, st));
    a.order = i32(p.order);
    a.ad = i32(p.ad);
  }
  const bool keep = ad && c.act != MOE_ACT_NONE;
  const float* mul = scales;
  if (dx && a.gshift >= 0) {
    const int groups = K / c.group_size;
    a.gs = reinterpret_cast<_Float16*>(w + p.gs);
    a.gs_low = (int64_t)N * groups;
    k_group_scales<<<N / 64, 256, 0, st>>>(scales, groups, f32(p.mul), reinterpret_cast<_Float16*>(w + p.gs), a.gs_low,
                                           scaled_parts<TX>() == 2);
    mul = f32(p.mul);
  }
  if (dx || keep) {
    DzArgs d{a, dy, pre, ldd, ldp, vec(dy, ldd), vec(pre, ldp), N, c.act == MOE_ACT_SWIGLU ? N / 2 : 0, c.act,
             dx ? mul : nullptr, keep ? f32(p.dz) : nullptr};
    if (c.act == MOE_ACT_NONE) dz_launch<TX, 0>(d, st);
    else if (c.act == MOE_ACT_SWIGLU) dz_launch<TX, 2>(d, st);
    else dz_launch<TX, 1>(d, st);
  }
  if (ad) {
    const void* m = keep ? w + p.dz : dy;  // dz, in fp32 by position or in the call's type by token
    const int64_t ldm = keep ? N : ldd;
    const int32_t* m_order = keep ? nullptr : a.order;
    const int vec_m = keep || vec(dy, ldd);
    // few: A and B as they are
    if (!few)
      MOE_TRY(launch_adapt_transpose(
          {a.n_ad, order.offsets, {{ad->b, N, a.R, w + p.bt}, {ad->a, a.R, K, dx ? w + p.at : nullptr}}}, elem, st));
    AdaptDown down{T, a.R, a.n_ad, db ? 2 : 1, few || adapt_few(T, a.R), 0, a.ad, order.n_runs, order.runs, ad->scale, {}};
    down.part[0] = {m, ldm, keep, vec_m, N, m_order, few ? ad->b : w + p.bt, few, f32(p.u), f32(p.ut)};
    down.part[1] = {x, ldx, 0, vec(x, ldx), K, a.order, ad->a, 0, f32(p.h), f32(p.ht)};
    MOE_TRY(launch_adapt_down(down, dtype, st));
    if (da || db) {
      AdaptOuter outer{T, a.R, a.n_ad, ids, order, {}};
      outer.part[0] = {m, ldm, keep, vec_m, N, 1, m_order, f32(p.h), f32(p.ht), f32(p.part), db};
      outer.part[1] = {x, ldx, 0, vec(x, ldx), K, 0, a.order, f32(p.u), f32(p.ut), f32(p.part_a), da};
      MOE_TRY(launch_adapt_outer(outer, dtype, st));
    }
    if (dx) {
      a.h = f32(p.u);
      a.ab = few ? ad->a : w + p.at;
    }
  }
  const int bits = c.weight_bits == 8 ? 8 : 4;
  if (dx && few) few_launch<TX>(a, bits, f32(p.sums), st);
  else if (dx) tiles_launch<TX>(a, bits, f32(p.sums), st);
#undef MOE_TRY
  return hipGetLastError();
}

}  // namespace

size_t linear_grad_ws_bytes(const moe_linear_config& c, const moe_adapters* ad, int64_t T) {
  return grad_plan(c, ad, T).total;
}

hipError_t launch_linear_grad(const moe_linear_config& c, const uint8_t* codes, const float* scales,
                              const moe_adapters* ad, const int32_t* ids, const void* x, int64_t ldx, int T, int dtype,
                              const void* pre, int64_t ldp, const void* dy, int64_t ldd, const void* res, int64_t ldr,
                              void* dx, int64_t ldg, void* da, void* db, void* ws, hipStream_t st) {
  const auto f = dtype == MOE_DTYPE_F32 ? run<float> : dtype == MOE_DTYPE_BF16 ? run<bf16_t> : run<_Float16>;
  return f(c, codes, scales, ad, ids, x, ldx, T, dtype, pre, ldp, dy, ldd, res, ldr, dx, ldg, da, db, ws, st);
}

}  // namespace moe
