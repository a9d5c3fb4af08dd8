// k_adapt.hip — low-rank adapters beside a product over weight codes: the first half s (A x) of what a token's adapter adds,
// the order of the tokens by adapter, and the gradients of A and B.
#include "linear_types.h"

namespace moe {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ order by adapter
// Positions: the tokens of adapter 0, of adapter 1, ..., those without one; ascending tokens in each. Every workgroup
// counts all tokens; wavefront w of a workgroup then places those of one adapter, 64 at a time by ballot, so the order is
// the same at every call. Workgroup 0 writes the gradients' table.
constexpr int kMaxAdapters = 1024;
constexpr int kOrderLds = 24576;  // tokens whose adapters fit LDS as 16-bit numbers

// exclusive prefix sum of one value for each of 1024 adapters and one more, v[i] of adapter 4 * tid + i; total returned
__device__ __forceinline__ int scan1024(int (&v)[4], int* s_wave) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = v[i];
    v[i] = sum;
    sum += c;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) s_wave[wave] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) before += s_wave[w];
    total += s_wave[w];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] += before + incl - sum;
  return total;
}

template <bool LDS>
__global__ __launch_bounds__(256) void k_adapt_order(const int32_t* __restrict__ ids, int T, int n, int32_t* __restrict__ order,
                                                     int32_t* __restrict__ pos_ad, AdaptTable table, int len) {
  __shared__ int s_count[kMaxAdapters + 1], s_first[kMaxAdapters + 1], s_wave[4];
  extern __shared__ int16_t s_ids[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e <= n; e += 256) s_count[e] = 0;
  __syncthreads();
  auto adapter = [&](int t) __attribute__((always_inline)) {
    const int id = ids ? ids[t] : 0;
    return (uint32_t)id < (uint32_t)n ? id : n;
  };
  constexpr int U = 8;
  for (int t0 = 0; t0 < T; t0 += 256 * U) {
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + 256 * u + tid;
      e[u] = t < T ? adapter(t) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e[u] >= 0) {
        if (LDS) s_ids[t0 + 256 * u + tid] = (int16_t)e[u];
        atomicAdd(&s_count[e[u]], 1);
      }
  }
  __syncthreads();
  int v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = 4 * tid + i < n ? s_count[4 * tid + i] : 0;
  const int with = scan1024(v, s_wave);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * tid + i < n) s_first[4 * tid + i] = v[i];
  if (tid == 0) s_first[n] = with;
  __syncthreads();

  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  const int e = blockIdx.x * 4 + wave;
  if (e <= n) {
    int pos = s_first[e];
    const int end = pos + s_count[e];
    for (int t0 = 0; t0 < T && pos < end; t0 += 256) {
      int id[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + 64 * u + lane;
        id[u] = t < T ? (LDS ? (int)s_ids[t] : adapter(t)) : -1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint64_t m = __ballot(id[u] == e);
        if (id[u] == e) {
          const int p = pos + __popcll(m & below);
          order[p] = t0 + 64 * u + lane;
          pos_ad[p] = e < n ? e : -1;
        }
        pos += __popcll(m);
      }
    }
  }
  if (blockIdx.x != 0 || !table.offsets) return;
  for (int i = tid; i <= n; i += 256) table.offsets[i] = s_first[i];
  int ch[4], sl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = 4 * tid + i < n ? (s_count[4 * tid + i] + len - 1) / len : 0;
    ch[i] = k;
    sl[i] = k > 1 ? k : 0;
  }
  const int chunks = scan1024(ch, s_wave);
  scan1024(sl, s_wave);
  if (tid == 0) *table.n_chunks = chunks;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = 4 * tid + i;
    if (a >= n) continue;
    const int p0 = s_first[a], p1 = p0 + s_count[a], k = (p1 - p0 + len - 1) / len;
    table.slot0[a] = sl[i];
    for (int j = 0; j < k; ++j)
      table.chunks[ch[i] + j] = AdaptChunk{a, p0 + j * len, min(p0 + (j + 1) * len, p1), k > 1 ? sl[i] + j : -1};
  }
}

// ------------------------------------------------------------ s (A x)
__device__ __forceinline__ int adapter_of(const AdaptDown& a, int p) {
  const int id = a.ad ? a.ad[p] : 0;
  return (uint32_t)id < (uint32_t)a.n_ad ? id : -1;
}
__device__ __forceinline__ void put_h(const AdaptDown& a, int p, int r, float v) {
  a.h[(size_t)p * a.R + r] = v;
  if (a.ht) a.ht[(size_t)r * a.ldt + p] = v;
}

// Few tokens: a workgroup takes a token and 4 rows of its A; its lanes share the columns, all loads in flight at once.
template <class TX>
__global__ __launch_bounds__(256) void k_adapt_dot(AdaptDown a) {
  __shared__ float s_sum[4][4];
  const int p = blockIdx.x, r0 = blockIdx.y * 4, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = adapter_of(a, p);
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (e >= 0) {
    const TX* x = static_cast<const TX*>(a.x) + (size_t)(a.order ? a.order[p] : p) * a.ldx;
    const TX* w = static_cast<const TX*>(a.a) + ((size_t)e * a.R + r0) * a.C;
#pragma unroll 4
    for (int g = tid; g < a.C / 8; g += 256) {
      Granule<TX> xg, wg[4];
      load8(x + g * 8, a.vec_x, xg);
#pragma unroll
      for (int i = 0; i < 4; ++i) load8(w + (size_t)i * a.C + g * 8, true, wg[i]);
      const f8v xv = granule_f32<TX>(xg);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f8v wv = granule_f32<TX>(wg[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i] = fmaf(xv[j], wv[j], v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v[i] += __shfl_xor(v[i], o);
  }
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[wave][i] = v[i];
  __syncthreads();
  if (tid < 4) {
    const float sum = s_sum[0][tid] + s_sum[1][tid] + s_sum[2][tid] + s_sum[3][tid];
    put_h(a, p, r0 + tid, e >= 0 ? a.scale[e] * sum : 0.0f);
  }
}

// More: 16 positions a workgroup, one product of all 16 for each adapter that they have (positions are in the order of
// their adapters, so it is mostly one), whose results go to the adapter's own positions only. Eight wavefronts share the
// columns. fp32 is multiplied in fp32, the others in their type, which is exact.
constexpr int kDownWaves = 8;
template <class TX, int RF>
__global__ __launch_bounds__(64 * kDownWaves) void k_adapt_down(AdaptDown a) {
  __shared__ float s_sum[kDownWaves][16][16 * RF + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int p0 = blockIdx.x * 16, p = min(p0 + i, a.T - 1);
  const int id = p0 + i < a.T ? adapter_of(a, p) : -1;
  const TX* x = static_cast<const TX*>(a.x) + (size_t)(a.order ? a.order[p] : p) * a.ldx + g * (sizeof(TX) == 4 ? 4 : 8);
  const int steps = a.C / 32, per = (steps + kDownWaves - 1) / kDownWaves;
  const int s0 = min(wave * per, steps), s1 = min(s0 + per, steps);
  uint32_t todo = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  const uint32_t have = todo;
  for (int k = tid; k < 16 * a.R; k += 64 * kDownWaves)
    if (p0 + k / a.R < a.T && !(have >> (k / a.R) & 1)) put_h(a, p0 + k / a.R, k % a.R, 0.0f);
  while (todo) {
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t mine = (uint32_t)__ballot(id == e) & 0xFFFFu;
    todo &= ~mine;
    const TX* w[RF];
    f4 acc[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      w[f] = static_cast<const TX*>(a.a) + ((size_t)e * a.R + min(16 * f + i, a.R - 1)) * a.C + g * (sizeof(TX) == 4 ? 4 : 8);
      acc[f] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
      if constexpr (std::is_same<TX, float>::value) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = s * 32 + h * 16;
          f4 xv;
          if (a.vec_x) xv = *reinterpret_cast<const f4*>(x + at);
          else xv = f4{x[at], x[at + 1], x[at + 2], x[at + 3]};
#pragma unroll
          for (int f = 0; f < RF; ++f) {
            const f4 wv = *reinterpret_cast<const f4*>(w[f] + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[f] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[j], wv[j], acc[f], 0, 0, 0);
          }
        }
      } else {
        Granule<TX> xg, wg;
        load8(x + s * 32, a.vec_x, xg);
#pragma unroll
        for (int f = 0; f < RF; ++f) {
          load8(w[f] + s * 32, true, wg);
          if constexpr (std::is_same<TX, bf16_t>::value)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, xg), __builtin_bit_cast(b8, wg), acc[f],
                                                             0, 0, 0);
          else
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, xg), __builtin_bit_cast(h8, wg), acc[f],
                                                            0, 0, 0);
        }
      }
    }
    // sum j of a lane: position 4 g + j, row l % 16
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) s_sum[wave][4 * g + j][16 * f + i] = acc[f][j];
    __syncthreads();
    const float scale = a.scale[e];
    for (int k = tid; k < 16 * a.R; k += 64 * kDownWaves) {
      const int q = k / a.R, r = k % a.R;
      if (!(mine >> q & 1)) continue;
      float v = s_sum[0][q][r];
#pragma unroll
      for (int u = 1; u < kDownWaves; ++u) v += s_sum[u][q][r];
      put_h(a, p0 + q, r, scale * v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ gradients of A and B
// out[r][c] = sum over an adapter's positions of v[p][r] m[p][c]; a wavefront takes 32 rows r (fewer where R is less) by
// 128 columns, a workgroup four of them and a run of positions. Positions are what is summed over, and neither m nor v
// has neighbouring ones in memory: a lane loads 8 columns of each of 8 positions and exchanges halves of words between
// two positions, which gives the operands of 8 products (column l + j of every eight columns in product j). v is read
// transposed. As in the product's epilogue v has two bf16 parts, bf16 m one and fp16 m two. fp32 is multiplied as it is,
// 4 columns a lane.
template <class TX>
__device__ __forceinline__ void put_outer(const AdaptOuter& a, const AdaptChunk& ch, int r, int c, const float* v, int rstep,
                                          int count) {
  // `count` neighbours, along r (rstep 1) or along c (0)
  if (ch.slot >= 0) {
    float* o = a.part + ((size_t)ch.slot * a.R + r) * a.C + c;
    for (int k = 0; k < count; ++k) o[rstep ? (size_t)k * a.C : (size_t)k] = v[k];
  } else {
    TX* o = static_cast<TX*>(a.out) +
            (a.rows ? ((size_t)ch.e * a.C + c) * a.R + r : ((size_t)ch.e * a.R + r) * a.C + c);
    const size_t step = (a.rows != 0) == (rstep != 0) ? 1 : (a.rows ? a.R : a.C);
    for (int k = 0; k < count; ++k) o[k * step] = from_f32<TX>(v[k]);
  }
}

template <class TX, int RF>
__global__ __launch_bounds__(256) void k_adapt_outer(AdaptOuter a) {
  if ((int)blockIdx.y >= *a.table.n_chunks) return;
  const AdaptChunk ch = a.table.chunks[blockIdx.y];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.z * 16 * RF;
  if constexpr (std::is_same<TX, float>::value) {
    const int c0 = (blockIdx.x * 4 + wave) * 64 + 4 * i;
    const bool in = c0 < a.C;
    f4 acc[RF][4];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[f][k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int p = ch.p0; p < ch.p1; p += 4) {
      const int t = p + g;
      f4 m = {0.0f, 0.0f, 0.0f, 0.0f};
      float v[RF];
#pragma unroll
      for (int f = 0; f < RF; ++f) v[f] = 0.0f;
      if (t < ch.p1) {
        if (in) {
          const float* q = static_cast<const float*>(a.m) + (size_t)(a.order ? a.order[t] : t) * a.ldm + c0;
          if (a.vec_m) m = *reinterpret_cast<const f4*>(q);
          else m = f4{q[0], q[1], q[2], q[3]};
        }
#pragma unroll
        for (int f = 0; f < RF; ++f) v[f] = a.v[(size_t)t * a.R + min(r0 + 16 * f + i, a.R - 1)];
      }
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[f][k] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[f], m[k], acc[f][k], 0, 0, 0);
    }
    if (!in) return;
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + 16 * f + 4 * g + j;
        if (r >= a.R) continue;
        const float o[4] = {acc[f][0][j], acc[f][1][j], acc[f][2][j], acc[f][3][j]};
        put_outer<TX>(a, ch, r, c0, o, 0, 4);
      }
  } else {
    constexpr int MP = std::is_same<TX, bf16_t>::value ? 1 : 2;  // parts of m
    const int c0 = (blockIdx.x * 4 + wave) * 128 + 8 * i;
    const bool in = c0 < a.C;
    f4 acc[RF][8];
#pragma unroll
    for (int f = 0; f < RF; ++f)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[f][k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = ch.p0 & ~7; p < ch.p1; p += 32) {
      const int t0 = p + 8 * g;
      Granule<TX> m[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int t = t0 + j;
        m[j] = Granule<TX>{};
        if (in && t >= ch.p0 && t < ch.p1)
          load8(static_cast<const TX*>(a.m) + (size_t)(a.order ? a.order[t] : t) * a.ldm + c0, a.vec_m, m[j]);
      }
      b8 vh[RF], vl[RF];
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        f8v v = {};
        if (t0 < ch.p1) {
          v = *reinterpret_cast<const f8v*>(a.vt + (size_t)min(r0 + 16 * f + i, a.R - 1) * a.ldt + t0);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = t0 + j >= ch.p0 && t0 + j < ch.p1 ? v[j] : 0.0f;
        }
        split_bf16(v, vh[f], vl[f]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // column 2 k + half
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = __builtin_amdgcn_perm(m[2 * q + 1].w[k], m[2 * q].w[k], half ? 0x07060302u : 0x05040100u);
          b8 mh, ml;
          if constexpr (MP == 1) {
            __builtin_memcpy(&mh, w, 16);
          } else {
            Granule<TX> t;
            __builtin_memcpy(&t, w, 16);
            split_bf16(granule_f32<TX>(t), mh, ml);
          }
#pragma unroll
          for (int f = 0; f < RF; ++f) {
            f4& c = acc[f][2 * k + half];
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vl[f], mh, c, 0, 0, 0);
            if constexpr (MP == 2) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vh[f], ml, c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vh[f], mh, c, 0, 0, 0);
          }
        }
    }
    if (!in) return;
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      if (a.rows && ch.slot < 0) {
        const int r = r0 + 16 * f + 4 * g;
        if (r < a.R)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float o[4] = {acc[f][k][0], acc[f][k][1], acc[f][k][2], acc[f][k][3]};
            put_outer<TX>(a, ch, r, c0 + k, o, 1, 4);
          }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + 16 * f + 4 * g + j;
          if (r >= a.R) continue;
          const float o[8] = {acc[f][0][j], acc[f][1][j], acc[f][2][j], acc[f][3][j],
                              acc[f][4][j], acc[f][5][j], acc[f][6][j], acc[f][7][j]};
          put_outer<TX>(a, ch, r, c0, o, 0, 8);
        }
      }
    }
  }
}

// Adapters of several runs: their partial sums in ascending order. Adapters without tokens: zeros.
template <class TX>
__global__ __launch_bounds__(256) void k_adapt_join(AdaptOuter a, int len) {
  const int c = blockIdx.x * 256 + threadIdx.x, r0 = blockIdx.z * 8, e = blockIdx.y;
  const int n = (a.table.offsets[e + 1] - a.table.offsets[e] + len - 1) / len;
  if (n == 1 || c >= a.C) return;
  float v[8] = {};
  const int slot = a.table.slot0[e];
  for (int k = 0; k < n; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += a.part[((size_t)(slot + k) * a.R + r0 + j) * a.C + c];
  TX* o = static_cast<TX*>(a.out) + (a.rows ? ((size_t)e * a.C + c) * a.R + r0 : ((size_t)e * a.R + r0) * a.C + c);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[a.rows ? (size_t)j : (size_t)j * a.C] = from_f32<TX>(v[j]);
}

template <class V>
__global__ __launch_bounds__(256) void k_adapt_transpose(const V* __restrict__ in, int M, int Q,
                                                         const int32_t* __restrict__ offsets, V* __restrict__ out) {
  __shared__ V s[32][33];
  const int e = blockIdx.z;
  if (offsets[e + 1] == offsets[e]) return;
  const int q0 = blockIdx.x * 32, m0 = blockIdx.y * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const size_t base = (size_t)e * M * Q;
  for (int k = ty; k < 32; k += 8)
    if (m0 + k < M && q0 + tx < Q) s[k][tx] = in[base + (size_t)(m0 + k) * Q + q0 + tx];
  __syncthreads();
  for (int k = ty; k < 32; k += 8)
    if (q0 + k < Q && m0 + tx < M) out[base + (size_t)(q0 + k) * M + m0 + tx] = s[tx][k];
}

template <class TX>
void down_launch(const AdaptDown& a, hipStream_t st) {
  // a workgroup for each token and four rows, or 16 tokens a workgroup
  if ((int64_t)a.T * a.R <= 4096) {
    k_adapt_dot<TX><<<dim3(a.T, a.R / 4), 256, 0, st>>>(a);
    return;
  }
  const int grid = (a.T + 15) / 16;
  if (a.R <= 16) k_adapt_down<TX, 1><<<grid, 64 * kDownWaves, 0, st>>>(a);
  else if (a.R <= 32) k_adapt_down<TX, 2><<<grid, 64 * kDownWaves, 0, st>>>(a);
  else if (a.R <= 64) k_adapt_down<TX, 4><<<grid, 64 * kDownWaves, 0, st>>>(a);
  else k_adapt_down<TX, 8><<<grid, 64 * kDownWaves, 0, st>>>(a);
}
template <class TX>
void outer_launch(const AdaptOuter& a, hipStream_t st) {
  const int per = std::is_same<TX, float>::value ? 256 : 512, cols = (a.C + per - 1) / per;
  const int chunks = (int)adapt_max_chunks(a.T, a.n_ad);
  if (a.R <= 16) k_adapt_outer<TX, 1><<<dim3(cols, chunks, 1), 256, 0, st>>>(a);
  else k_adapt_outer<TX, 2><<<dim3(cols, chunks, (a.R + 31) / 32), 256, 0, st>>>(a);
  k_adapt_join<TX><<<dim3((a.C + 255) / 256, a.n_ad, a.R / 8), 256, 0, st>>>(a, adapt_chunk_len(a.T));
}

}  // namespace

hipError_t launch_adapt_order(const int32_t* ids, int T, int n_ad, int32_t* order, int32_t* pos_ad, hipStream_t st,
                              const AdaptTable* table) {
  const AdaptTable t = table ? *table : AdaptTable{};
  const int grid = n_ad / 4 + 1, len = adapt_chunk_len(T);  // one more than the adapters: the tokens without one
  if (T <= kOrderLds) k_adapt_order<true><<<grid, 256, (size_t)T * 2, st>>>(ids, T, n_ad, order, pos_ad, t, len);
  else k_adapt_order<false><<<grid, 256, 0, st>>>(ids, T, n_ad, order, pos_ad, t, len);
  return hipGetLastError();
}
hipError_t launch_adapt_down(const AdaptDown& a, int dtype, hipStream_t st) {
  if (dtype == MOE_DTYPE_F32) down_launch<float>(a, st);
  else if (dtype == MOE_DTYPE_BF16) down_launch<bf16_t>(a, st);
  else down_launch<_Float16>(a, st);
  return hipGetLastError();
}
hipError_t launch_adapt_outer(const AdaptOuter& a, int dtype, hipStream_t st) {
  if (dtype == MOE_DTYPE_F32) outer_launch<float>(a, st);
  else if (dtype == MOE_DTYPE_BF16) outer_launch<bf16_t>(a, st);
  else outer_launch<_Float16>(a, st);
  return hipGetLastError();
}
hipError_t launch_adapt_transpose(const void* in, int n, int M, int Q, int elem, const int32_t* offsets, void* out,
                                  hipStream_t st) {
  const dim3 grid((Q + 31) / 32, (M + 31) / 32, n);
  if (elem == 4)
    k_adapt_transpose<<<grid, 256, 0, st>>>(static_cast<const uint32_t*>(in), M, Q, offsets, static_cast<uint32_t*>(out));
  else
    k_adapt_transpose<<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(in), M, Q, offsets, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

}  // namespace moe
