// k_linear_grad.hip — gradients of y = act(W x + b + s B (A x)) for frozen codes W: with dz = dy act'(z),
//   dx = W^T dz + s A^T (B^T dz),  dB = sum over tokens of dz (s A x)^T,  dA = sum over tokens of (s B^T dz) x^T.
// W^T dz runs in the product's tiles, summing over the weight rows. Row scales are multiplied into dz, in fp32 before its
// one rounding to fp16 (relative 2^-12; fp32 gradients keep two halves, 2^-23). Group scales differ along a row: the power
// of two of a row's largest is multiplied into dz, without loss, what is left of them, at most 1, into the codes, as fp16
// (relative 2^-11, or 2^-25 of the row's largest for scales that are less than 2^-14 of it; fp32 gradients keep two parts,
// 2^-19). dz is kept in the call's type for the adapters' sums, as autograd would hand it on.
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
  void* dz;              // [T][N] by position, or nullptr
};

template <class TX>
__device__ __forceinline__ f8v dz8(const DzArgs& d, int64_t t, int n) {
  Granule<TX> g, z, u;
  const int at = d.half && n >= d.half ? n - d.half : n;
  load8(static_cast<const TX*>(d.dy) + t * d.ldd + at, d.vec_d, g);
  f8v v = granule_f32<TX>(g);
  if (d.act == MOE_ACT_NONE) return v;
  const TX* p = static_cast<const TX*>(d.pre) + t * d.ldp;
  load8(p + at, d.vec_p, z);
  const f8v zv = granule_f32<TX>(z);
  if (!d.half) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= slope(zv[i], d.act);
  } else if (n < d.half) {
    load8(p + d.half + at, d.vec_p, u);
    const f8v uv = granule_f32<TX>(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * uv[i] * slope(zv[i], MOE_ACT_SILU);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, miss;
      sigmoid2(zv[i], s, miss);
      v[i] *= zv[i] < -1e9f ? 0.0f : zv[i] * s;
    }
  }
  return v;
}

// As k_linear_x, from dz: 8 positions a workgroup, the largest of a token first.
template <class TX>
__global__ __launch_bounds__(8 * kPrepLanes) void k_linear_dz(DzArgs d) {
  constexpr int kRounds = 4;  // granules whose values stay in registers
  __shared__ uint32_t s_max[16][8];
  const LinearArgs& a = d.a;
  const int tk = threadIdx.x & 7, g0 = threadIdx.x >> 3;
  const int p = blockIdx.x * 8 + tk;
  const bool in = p < a.T;
  const int64_t t = in ? token_of(a, p) : 0;
  const int ng = in ? d.N / 8 : 0;
  f8v v[kRounds];
  uint32_t m = 0;
  auto scaled = [&](int g, bool keep) __attribute__((always_inline)) {
    f8v w = dz8<TX>(d, t, g * 8);
    if (keep && d.dz) {
      TX o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = from_f32<TX>(w[i]);
      Granule<TX> q;
      __builtin_memcpy(&q, o, sizeof(q));
      u4v* to = reinterpret_cast<u4v*>(static_cast<TX*>(d.dz) + (size_t)p * d.N + g * 8);
#pragma unroll
      for (int i = 0; i < (int)sizeof(TX) / 2; ++i) to[i] = u4v{q.w[4 * i], q.w[4 * i + 1], q.w[4 * i + 2], q.w[4 * i + 3]};
    }
    if (d.mul) {
      const f8v s = *reinterpret_cast<const f8v*>(d.mul + g * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] *= s[i];
    }
    return w;
  };
  auto largest = [&](const f8v& w) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(w[i]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int k = 0; k < kRounds; ++k)
    if (g0 + k * kPrepLanes < ng) {
      v[k] = scaled(g0 + k * kPrepLanes, true);
      largest(v[k]);
    }
  for (int g = g0 + kRounds * kPrepLanes; g < ng; g += kPrepLanes) largest(scaled(g, true));
  if (!d.mul) return;
#pragma unroll
  for (int o = 8; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  if ((threadIdx.x & 63) < 8) s_max[threadIdx.x >> 6][tk] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, s_max[i][tk]);
  const bool finite = m < 0x7F800000u;
  const int sh = scale_shift(m);
  if (in && g0 == 0) a.sh[p] = sh;
  const size_t base = (size_t)(p >> 5) * a.nbp * 1024 + (size_t)(p & 31) * 8;
  auto store = [&](int g, f8v w) __attribute__((always_inline)) {
    h8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = ldexpf(w[(i >> 1) + 4 * (i & 1)], sh);
      if (!finite && fabsf(x) < INFINITY) x = fminf(fmaxf(x, -65504.0f), 65504.0f);
      hi[i] = (_Float16)x;
      lo[i] = fabsf(x) < INFINITY ? (_Float16)(x - (float)hi[i]) : (_Float16)0.0f;
    }
    const size_t at = base + (size_t)g * 256;
    *reinterpret_cast<h8*>(a.xh + at) = hi;
    if (std::is_same<TX, float>::value) *reinterpret_cast<h8*>(a.xl + at) = lo;
  };
#pragma unroll
  for (int k = 0; k < kRounds; ++k)
    if (g0 + k * kPrepLanes < d.N / 8) store(g0 + k * kPrepLanes, in ? v[k] : f8v{});
  for (int g = g0 + kRounds * kPrepLanes; g < d.N / 8; g += kPrepLanes) store(g, in ? scaled(g, false) : f8v{});
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
  const int e = m > 0.0f && m < INFINITY ? __builtin_amdgcn_frexp_expf(m) : 0;  // m = f 2^e, f in [1/2, 1)
  if (wave == 0) mul[blockIdx.x * 64 + lane] = ldexpf(1.0f, e);
  // place of row l in the order of the codes: eight rows 0 4 1 5 2 6 3 7
  const int r = lane & 7, at = (lane & ~7) + (r < 4 ? 2 * r : 2 * (r - 4) + 1);
  for (int g = wave; g < groups; g += 4) {
    const float v = ldexpf(s[(size_t)g * 64], -e);
    const size_t o = ((size_t)blockIdx.x * groups + g) * 64 + at;
    if (!low) {
      gs[o] = (_Float16)v;
    } else {  // eight bits, whose product with a code is exact, and the rest
      const float hi = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
      gs[o] = (_Float16)hi;
      gs[gs_low + o] = (_Float16)(v - (float)(_Float16)hi);
    }
  }
}

// ------------------------------------------------------------ the whole
struct GradPlan {
  LinearPlan z;
  size_t mul, gs, dz, order, ad, offsets, slot0, n_chunks, chunks, h, ht, u, ut, at, bt, part, total;
  int ldt;
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
  p.ldt = (int)((T + 7) & ~7);
  if (ad) {
    const size_t R = ad->rank, n = ad->n_adapters, N = c.rows, K = c.cols;
    p.dz = take(c.act != MOE_ACT_NONE ? T * N * 4 : 0);
    p.order = take(T * 4);
    p.ad = take(T * 4);
    p.offsets = take((n + 1) * 4);
    p.slot0 = take(n * 4);
    p.n_chunks = take(4);
    p.chunks = take(sizeof(AdaptChunk) * (size_t)adapt_max_chunks(T, (int)n));
    p.h = take(T * R * 4);
    p.ht = take(p.ldt * R * 4);
    p.u = take(T * R * 4);
    p.ut = take(p.ldt * R * 4);
    p.at = take(n * R * K * 4);
    p.bt = take(n * R * N * 4);
    p.part = take((size_t)kAdaptSlots * R * std::max(N, K) * 4);
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

  AdaptTable table{};
  if (ad) {
    table = AdaptTable{i32(p.offsets), i32(p.slot0), i32(p.n_chunks), reinterpret_cast<AdaptChunk*>(w + p.chunks)};
    MOE_TRY(launch_adapt_order(ids, T, ad->n_adapters, i32(p.order), i32(p.ad), st, &table));
    a.order = i32(p.order);
    a.ad = i32(p.ad);
    a.n_ad = ad->n_adapters;
    a.R = ad->rank;
  }
  const bool keep = ad && c.act != MOE_ACT_NONE;
  const float* mul = scales;
  if (dx && a.gshift >= 0) {
    const int groups = K / c.group_size;
    a.gs = reinterpret_cast<_Float16*>(w + p.gs);
    a.gs_low = (int64_t)N * groups;
    k_group_scales<<<N / 64, 256, 0, st>>>(scales, groups, f32(p.mul), reinterpret_cast<_Float16*>(w + p.gs), a.gs_low,
                                           elem == 4);
    mul = f32(p.mul);
  }
  if (dx || keep) {
    DzArgs d{a, dy, pre, ldd, ldp, vec(dy, ldd), vec(pre, ldp), N, c.act == MOE_ACT_SWIGLU ? N / 2 : 0, c.act,
             dx ? mul : nullptr, keep ? w + p.dz : nullptr};
    k_linear_dz<TX><<<(T + 31) / 32 * 4, 8 * kPrepLanes, 0, st>>>(d);
  }
  if (ad) {
    const void* m = keep ? w + p.dz : dy;  // dz, by position or by token
    const int64_t ldm = keep ? N : ldd;
    const int32_t* m_order = keep ? nullptr : a.order;
    MOE_TRY(launch_adapt_transpose(ad->b, a.n_ad, N, a.R, elem, table.offsets, w + p.bt, st));
    MOE_TRY(launch_adapt_down({m, ldm, vec(m, ldm), T, N, a.R, a.n_ad, m_order, a.ad, w + p.bt, ad->scale, f32(p.u),
                               f32(p.ut), p.ldt}, dtype, st));
    if (dx) {
      MOE_TRY(launch_adapt_transpose(ad->a, a.n_ad, a.R, K, elem, table.offsets, w + p.at, st));
      a.h = f32(p.u);
      a.ab = w + p.at;
    }
    if (db) {
      MOE_TRY(launch_adapt_down({x, ldx, vec(x, ldx), T, K, a.R, a.n_ad, a.order, a.ad, ad->a, ad->scale, f32(p.h),
                                 f32(p.ht), p.ldt}, dtype, st));
      MOE_TRY(launch_adapt_outer({m, ldm, vec(m, ldm), T, N, a.R, a.n_ad, 1, m_order, f32(p.h), f32(p.ht), p.ldt, table,
                                  f32(p.part), db}, dtype, st));
    }
    if (da)
      MOE_TRY(launch_adapt_outer({x, ldx, vec(x, ldx), T, K, a.R, a.n_ad, 0, a.order, f32(p.u), f32(p.ut), p.ldt, table,
                                  f32(p.part), da}, dtype, st));
  }
  if (dx) tiles_launch<TX>(a, c.weight_bits == 8 ? 8 : 4, st);
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
