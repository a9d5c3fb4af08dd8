// k_adapt.hip — low-rank adapters beside a product over weight codes: the first half s (A x) of what a token's adapter adds,
// the order of the tokens by adapter, and the gradients of A and B.
#include <algorithm>

#include "linear_types.h"

namespace moe {

namespace {

typedef f4v f4;

// ------------------------------------------------------------ order by adapter
// Positions: the tokens of adapter 0, of adapter 1, ..., those without one; ascending tokens in each. One workgroup: each
// of its 16 wavefronts takes a stretch of the tokens, counts their adapters and, after the counts are summed up, places
// them, 64 at a time. Lanes of one adapter find each other by ballots over the bits of its number, so the order is the
// same at every call and a step takes as long for 64 adapters as for one. 33 tokens 5.5 us, 2,048 7 to 8: latency of its
// barriers and of the loads of ids.
constexpr int kMaxAdapters = 1024, kOrderWaves = 16;

// exclusive prefix sum over 1024 threads; the total of all
__device__ __forceinline__ int scan1024(int& v, int* s_wave) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) s_wave[wave] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kOrderWaves; ++w) {
    if (w < wave) before += s_wave[w];
    total += s_wave[w];
  }
  __syncthreads();
  v = before + incl - v;
  return total;
}

__global__ __launch_bounds__(64 * kOrderWaves) void k_adapt_order(const int32_t* __restrict__ ids, int T, int n, AdaptOrder out,
                                                                  int len) {
  __shared__ int s_at[kOrderWaves][kMaxAdapters + 1];  // counts, then the next position of each adapter and wavefront
  __shared__ int s_first[kMaxAdapters + 1], s_wave[kOrderWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bits = 32 - __builtin_clz(n);  // of 0 .. n
  const int per = ((T + kOrderWaves - 1) / kOrderWaves + 63) & ~63, t0 = wave * per, t1 = min(t0 + per, T);
  auto adapter = [&](int t) __attribute__((always_inline)) {
    const int id = ids && t < t1 ? ids[t] : 0;
    return (uint32_t)id < (uint32_t)n ? id : n;
  };
  constexpr int kHeld = 4;  // steps whose adapters stay in registers
  int held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = adapter(t0 + 64 * k + lane);
#pragma unroll
  for (int w = 0; w < kOrderWaves; ++w)
    for (int k = tid; k <= n; k += 64 * kOrderWaves) s_at[w][k] = 0;
  __syncthreads();
  auto same = [&](int e, bool in) __attribute__((always_inline)) {
    uint64_t m = __ballot(in);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      m &= e >> b & 1 ? set : ~set;
    }
    return m;
  };
  auto tally = [&](int t, int e) __attribute__((always_inline)) {
    const bool in = t + lane < t1;
    const uint64_t m = same(e, in);
    if (in && lane == __builtin_ctzll(m)) s_at[wave][e] += (int)__popcll(m);
    wave_sync();  // the next step's first lane of this adapter is another one
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (t0 + 64 * k < t1) tally(t0 + 64 * k, held[k]);
  for (int t = t0 + 64 * kHeld; t < t1; t += 64) tally(t, adapter(t + lane));
  __syncthreads();
  int count = 0;
  if (tid < n)
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) count += s_at[w][tid];
  int first = count;
  const int with = scan1024(first, s_wave);
  auto spread = [&](int e, int at) __attribute__((always_inline)) {
    s_first[e] = at;
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) {
      const int c = s_at[w][e];
      s_at[w][e] = at;
      at += c;
    }
  };
  if (tid < n) spread(tid, first);
  if (tid == 0) spread(n, with);
  __syncthreads();
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
  auto place = [&](int t, int e) __attribute__((always_inline)) {
    const bool in = t + lane < t1;
    const uint64_t m = same(e, in);
    const int at = s_at[wave][e];  // e is at most n, of lanes without a token too
    wave_sync();
    if (in) {
      const int p = at + (int)__popcll(m & below);
      if (lane == __builtin_ctzll(m)) s_at[wave][e] = at + (int)__popcll(m);
      out.order[p] = t + lane;
      out.ad[p] = e < n ? e : -1;
    }
    wave_sync();
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (t0 + 64 * k < t1) place(t0 + 64 * k, held[k]);
  for (int t = t0 + 64 * kHeld; t < t1; t += 64) place(t, adapter(t + lane));
  // runs of 16 positions, and the gradients' longer ones
  int runs = (count + 15) / 16, chunks = len > 0 ? (count + len - 1) / len : 0, slots = chunks > 1 ? chunks : 0;
  const int all_runs = scan1024(runs, s_wave);
  int both = chunks | slots << 16;  // at most 16 + 1024 and 32
  const int all_chunks = scan1024(both, s_wave) & 0xFFFF;
  chunks = both & 0xFFFF, slots = both >> 16;
  if (tid == 0) {
    *out.n_runs = all_runs;
    if (len > 0) *out.n_chunks = all_chunks;
  }
  if (tid < n) {
    s_at[0][tid] = runs;
    s_at[1][tid] = chunks;
    s_at[2][tid] = slots;
    if (len > 0) out.slot0[tid] = slots;
  }
  if (len > 0)
    for (int k = tid; k <= n; k += 64 * kOrderWaves) out.offsets[k] = s_first[k];
  __syncthreads();
  for (int e = wave; e < n; e += kOrderWaves) {
    const int p0 = s_first[e], p1 = s_first[e + 1];
    for (int p = p0 + 16 * lane, j = lane; p < p1; p += 1024, j += 64)
      out.runs[s_at[0][e] + j] = AdaptChunk{e, p, min(p + 16, p1), 0};
    if (len <= 0) continue;
    const int k = (p1 - p0 + len - 1) / len;  // at most 16
    if (lane < k)
      out.chunks[s_at[1][e] + lane] =
          AdaptChunk{e, p0 + lane * len, min(p0 + (lane + 1) * len, p1), k > 1 ? s_at[2][e] + lane : -1};
  }
}

// ------------------------------------------------------------ s (A x)
__device__ __forceinline__ int adapter_of(const AdaptDown& a, int p) {
  const int id = a.ad ? a.ad[p] : 0;
  return (uint32_t)id < (uint32_t)a.n_ad ? id : -1;
}
__device__ __forceinline__ void put_h(const AdaptDown& a, const AdaptDown::Part& d, int p, int r, float v) {
  d.h[(size_t)p * a.R + r] = v;
  if (d.ht) d.ht[((size_t)(p >> 3) * a.R + r) * 8 + (p & 7)] = v;
}

// Few tokens: a workgroup takes a token and 4 rows of its A; its lanes share the columns, all loads in flight at once.
// across: A lies as [C][R]. One token of 6144 columns, rank 16: 3.4 us, 191 of 2048, rank 8: 4.6; a launch and its loads.
template <class TX>
struct alignas(4 * sizeof(TX)) Four {
  TX v[4];
};
// a lane's share of the sums of rows r0 .. r0 + 3; TM: the type of x
template <class TX, class TM>
__device__ __forceinline__ void dot_rows(const AdaptDown& a, const AdaptDown::Part& d, int p, int e, int r0, float (&v)[4]) {
  const int tid = threadIdx.x;
  const TM* x = static_cast<const TM*>(d.x) + (size_t)(d.order ? d.order[p] : p) * d.ldx;
  if (d.across) {
    const TX* b = static_cast<const TX*>(d.a) + (size_t)e * a.R * d.C + r0;
#pragma unroll 8
    for (int c = tid; c < d.C; c += 256) {
      const float xv = to_f32<TM>(x[c]);
      const Four<TX> w = *reinterpret_cast<const Four<TX>*>(b + (size_t)c * a.R);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fmaf(xv, to_f32<TX>(w.v[i]), v[i]);
    }
  }
  const TX* w = static_cast<const TX*>(d.a) + ((size_t)e * a.R + r0) * d.C;
#pragma unroll 4
  for (int g = tid; g < d.C / 8 && !d.across; g += 256) {
    Granule<TM> xg;
    Granule<TX> wg[4];
    load8(x + g * 8, d.vec_x, xg);
#pragma unroll
    for (int i = 0; i < 4; ++i) load8(w + (size_t)i * d.C + g * 8, true, wg[i]);
    const f8v xv = granule_f32<TM>(xg);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f8v wv = granule_f32<TX>(wg[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i] = fmaf(xv[j], wv[j], v[i]);
    }
  }
}

template <class TX>
__global__ __launch_bounds__(256) void k_adapt_dot(AdaptDown a) {
  __shared__ float s_sum[4][4];
  const AdaptDown::Part& d = a.part[blockIdx.z];
  const int p = blockIdx.x, r0 = blockIdx.y * 4, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = adapter_of(a, p);
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (e >= 0) {
    if (!std::is_same<TX, float>::value && d.f32) dot_rows<TX, float>(a, d, p, e, r0, v);
    else dot_rows<TX, TX>(a, d, p, e, r0, v);
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
    put_h(a, d, p, r0 + tid, e >= 0 ? a.scale[e] * sum : 0.0f);
  }
}

// More: a run of up to 16 positions of one adapter and 16 RF rows a workgroup; its wavefronts share the columns, each with
// the loads of several steps (128 bytes of every row) in flight. Eight neighbouring lanes load a row's 128 bytes; the
// operands, a row a lane, come from LDS: loaded in the operands' order, where neighbouring lanes are in different rows, a
// load takes four times as long (14 us for any number of runs up to 128, rows of 6144 bf16; 8 us so where they are in the
// caches and 11 where not, 2,048 tokens of rank 32 14 to 15.5). Latency bounds it: run, token, row, columns are loaded one
// after the other. fp32 is multiplied in fp32 (by 16-bit A or B too, for a kept dz), the others in their type, which is exact.
constexpr int kDownWaves = 8;
template <class TX>
__device__ __forceinline__ u4v load_16(const TX* p, bool vec) {
  if (vec) return *reinterpret_cast<const u4v*>(p);
  TX t[16 / sizeof(TX)];
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(TX)); ++i) t[i] = p[i];
  return __builtin_bit_cast(u4v, t);
}
template <class TX>
__device__ __forceinline__ f4 mul_16(const u4v& x, const u4v& w, f4 c) {
  if constexpr (std::is_same<TX, float>::value) {
    const f4 xv = __builtin_bit_cast(f4, x), wv = __builtin_bit_cast(f4, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[j], wv[j], c, 0, 0, 0);
    return c;
  } else if constexpr (std::is_same<TX, bf16_t>::value) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, x), __builtin_bit_cast(b8, w), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, x), __builtin_bit_cast(h8, w), c, 0, 0, 0);
  }
}

// as many elements as 16 bytes of TM hold, as TM
template <class TX, class TM>
__device__ __forceinline__ u4v load_as(const TX* p) {
  if constexpr (std::is_same<TX, TM>::value) return load_16<TX>(p, true);
  const Four<TX> q = *reinterpret_cast<const Four<TX>*>(p);
  return __builtin_bit_cast(u4v, f4{to_f32<TX>(q.v[0]), to_f32<TX>(q.v[1]), to_f32<TX>(q.v[2]), to_f32<TX>(q.v[3])});
}

template <int RF>
constexpr size_t down_lds() {
  return std::max<size_t>((size_t)kDownWaves * (1 + RF) * 2048, sizeof(float) * kDownWaves * 16 * (16 * RF + 4));
}
// TM: the type of x, in which the products are taken; s_mem: a wavefront's rows of a step, [1 + RF][16][128 bytes], later the
// sums, [wavefronts][16][kSum]
template <class TX, class TM, int RF>
__device__ __forceinline__ void down_run(const AdaptDown& a, const AdaptDown::Part& d, const AdaptChunk& run, char* s_mem) {
  constexpr int kChunk = 16 / sizeof(TM), kStep = 8 * kChunk, U = RF == 1 ? 4 : 3;  // columns; steps at once
  constexpr int kSum = 16 * RF + 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, i = lane & 15, g = lane >> 4;
  const int r0 = blockIdx.y * 16 * RF, rows = min(16 * RF, a.R - r0);
  const int steps = (d.C + kStep - 1) / kStep, per = (steps + kDownWaves - 1) / kDownWaves;
  const int s0 = min(wave * per, steps), s1 = min(s0 + per, steps);
  // lane: row lane / 8 (and 8 more), chunk lane % 8, which goes to place chunk ^ row % 8, so that no two lanes that read
  // at a time meet in a bank
  const int chunk = (lane & 7) ^ (lane >> 3);
  const TM* x[2];
  const TX* w[RF][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int q = 8 * k + (lane >> 3), p = min(run.p0 + q, run.p1 - 1);
    x[k] = static_cast<const TM*>(d.x) + (size_t)(d.order ? d.order[p] : p) * d.ldx + chunk * kChunk;
#pragma unroll
    for (int f = 0; f < RF; ++f)
      w[f][k] = static_cast<const TX*>(d.a) + ((size_t)run.e * a.R + r0 + min(16 * f + q, rows - 1)) * d.C + chunk * kChunk;
  }
  f4 acc[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) acc[f] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  u4v* s_row = reinterpret_cast<u4v*>(s_mem) + wave * (1 + RF) * 128;
  for (int s = s0; s < s1; s += U) {
    u4v xv[U][2], wv[U][RF][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(s + u, s1 - 1) * kStep, c = at + chunk * kChunk < d.C ? at : -chunk * kChunk;  // they may end at half a step
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        xv[u][k] = load_16(x[k] + c, d.vec_x);
#pragma unroll
        for (int f = 0; f < RF; ++f) wv[u][f][k] = load_as<TX, TM>(w[f][k] + c);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= s1) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s_row[64 * k + lane] = xv[u][k];
#pragma unroll
        for (int f = 0; f < RF; ++f) s_row[128 * (1 + f) + 64 * k + lane] = wv[u][f][k];
      }
      wave_sync();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if ((s + u) * kStep + 4 * h * kChunk >= d.C) break;
        const int from = i * 8 + ((4 * h + g) ^ (i & 7));
        const u4v xf = s_row[from];
#pragma unroll
        for (int f = 0; f < RF; ++f) acc[f] = mul_16<TM>(xf, s_row[128 * (1 + f) + from], acc[f]);
      }
      wave_sync();
    }
  }
  // sum j of a lane: position 4 g + j, row l % 16
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(s_mem);
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j) s_sum[(wave * 16 + 4 * g + j) * kSum + 16 * f + i] = acc[f][j];
  __syncthreads();
  const float scale = a.scale[run.e];
  for (int k = tid; k < (run.p1 - run.p0) * rows; k += 64 * kDownWaves) {
    const int q = k / rows, r = k % rows, at = run.p0 + q;
    float v = s_sum[q * kSum + r];
#pragma unroll
    for (int u = 1; u < kDownWaves; ++u) v += s_sum[(u * 16 + q) * kSum + r];
    put_h(a, d, a.by_token && d.order ? d.order[at] : at, r0 + r, scale * v);
  }
}

template <class TX, int RF>
__global__ __launch_bounds__(64 * kDownWaves, 4) void k_adapt_down(AdaptDown a) {
  __shared__ __align__(16) char s_mem[down_lds<RF>()];
  const AdaptDown::Part& d = a.part[blockIdx.z];
  AdaptChunk run{0, (int)blockIdx.x * 16, min((int)blockIdx.x * 16 + 16, a.T), 0};  // the only adapter, whoever has it
  if (a.runs) {
    if ((int)blockIdx.x >= *a.n_runs) return;
    run = a.runs[blockIdx.x];
  }
  if (!std::is_same<TX, float>::value && d.f32) down_run<TX, float, RF>(a, d, run, s_mem);
  else down_run<TX, TX, RF>(a, d, run, s_mem);
}

// ------------------------------------------------------------ gradients of A and B
// out[r][c] = sum over an adapter's positions of v[p][r] m[p][c]; a workgroup takes 32 rows r (fewer where R is less) by
// 128 columns and a run of positions, of which each of its four wavefronts takes a part; both gradients in one launch. Positions are what is
// summed over, and neither m nor v has neighbouring ones in memory: a lane loads 8 columns of each of 8 positions and
// exchanges halves of words between two positions, which gives the operands of 8 products (column l + j of every eight
// columns in product j). v comes with eight
// positions of a row next to each other. As in the product's epilogue v has two bf16 parts, bf16 m one and fp16 m
// two, and the product of the low ones is left out. fp32 (a kept dz too) is multiplied as it is, 4 columns a lane. 2,000 tokens of four adapters, rank 32, 4096 columns of
// fp32 and 6144 of bf16: 20.4 us for 57 MB, 16.0 for 41 with both in bf16; two workgroups a compute unit fit the registers, and each waits for chunk, order and rows in turn.
__device__ __forceinline__ size_t outer_at(const AdaptOuter& a, const AdaptOuter::Part& d, int e, int r, int c) {
  return d.rows ? ((size_t)e * d.C + c) * a.R + r : ((size_t)e * a.R + r) * d.C + c;
}

// The positions of a run that this one of four wavefronts takes, cut at multiples of 8.
__device__ __forceinline__ void wave_part(const AdaptChunk& ch, int& w0, int& w1) {
  const int wave = threadIdx.x >> 6, begin = ch.p0 & ~7, per = ((ch.p1 - begin + 31) / 32) * 8;
  w0 = max(min(begin + wave * per, ch.p1), ch.p0);
  w1 = max(min(begin + (wave + 1) * per, ch.p1), ch.p0);
}

// FEW: positions are tokens, at most 64, and those that count are bits of `mine`.
template <class TX, int RF, bool FEW>
__device__ __forceinline__ void outer_16(const AdaptOuter& a, const AdaptOuter::Part& d, const AdaptChunk& ch, uint64_t mine,
                                         int c_group, int r0, float* s_sum) {
  int w0, w1;  // this wavefront's positions
  wave_part(ch, w0, w1);
  auto counts = [&](int t) __attribute__((always_inline)) { return t >= w0 && t < w1 && (!FEW || (mine >> t & 1)); };
  constexpr int MP = std::is_same<TX, bf16_t>::value ? 1 : 2;  // parts of m
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, c0 = c_group + 8 * i;
  const bool in = c0 < d.C;
  f4 acc[RF][8];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[f][k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  const float* vt[RF];
#pragma unroll
  for (int f = 0; f < RF; ++f) vt[f] = d.vt + (size_t)min(r0 + 16 * f + i, a.R - 1) * 8;
  const int begin = w0 & ~7, last = max(w1 - 1, 0) & ~7;
  Granule<TX> mn[8];
  f8v vn[RF];
  // Rows of m two steps ahead. Positions outside the part take the row of its first: v is 0 there, and what that row holds
  // is in the sum anyway, so that the loads need no conditions.
  int row[8];
  const int any = min(w0, max(w1 - 1, 0)), row0 = !FEW && d.order ? d.order[any] : any;
  const TX* m_col = static_cast<const TX*>(d.m) + min(c0, d.C - 8);
  auto rows_of = [&](int p) __attribute__((always_inline)) {
    const int t0 = p + 8 * g;
    if (!FEW && d.order) {
      const i4v* o = reinterpret_cast<const i4v*>(d.order + max(min(t0, last), begin));
      const i4v lo = o[0], hi = o[1];
#pragma unroll
      for (int j = 0; j < 8; ++j) row[j] = counts(t0 + j) ? (j < 4 ? lo[j & 3] : hi[j & 3]) : row0;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) row[j] = counts(t0 + j) ? t0 + j : row0;
    }
  };
  auto fetch = [&](int p) __attribute__((always_inline)) {
    const int t0 = p + 8 * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (FEW) mn[j] = Granule<TX>{};
      if (!FEW || counts(t0 + j)) load8(m_col + (size_t)row[j] * d.ldm, d.vec_m, mn[j]);
    }
#pragma unroll
    for (int f = 0; f < RF; ++f) vn[f] = *reinterpret_cast<const f8v*>(vt[f] + (size_t)min(t0, last) * a.R);
  };
  rows_of(begin);
  fetch(begin);
  rows_of(begin + 32);
  for (int p = begin; p < w1; p += 32) {
    Granule<TX> m[8];
    b8 vh[RF], vl[RF];
    const int t0 = p + 8 * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = mn[j];
#pragma unroll
    for (int f = 0; f < RF; ++f) {
      f8v v = vn[f];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = counts(t0 + j) ? v[j] : 0.0f;
      split_bf16(v, vh[f], vl[f]);
    }
    fetch(p + 32);
    rows_of(p + 64);
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
  // the wavefronts' sums through LDS, [wavefront][f][k][j][lane]
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) s_sum[(((wave * RF + f) * 8 + k) * 4 + j) * 64 + lane] = acc[f][k][j];
  __syncthreads();
  auto total = [&](int f, int k, int j) __attribute__((always_inline)) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += s_sum[(((w * RF + f) * 8 + k) * 4 + j) * 64 + lane];
    return v;
  };
  if (!in) return;
  struct alignas(16) Eight {
    TX v[8];
  };
  struct alignas(8) Quad4 {
    TX v[4];
  };
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int r = r0 + 16 * f + 4 * g;  // and three more
    if (r >= a.R) continue;
    if (d.rows && ch.slot < 0) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int k = 2 * wave + kk;
        Quad4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = from_f32<TX>(total(f, k, j));
        *reinterpret_cast<Quad4*>(static_cast<TX*>(d.out) + outer_at(a, d, ch.e, r, c0 + k)) = o;
      }
    } else {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = total(f, k, wave);
      if (ch.slot >= 0) {
        f4* o = reinterpret_cast<f4*>(d.part + ((size_t)ch.slot * a.R + r + wave) * d.C + c0);
        o[0] = f4{v[0], v[1], v[2], v[3]};
        o[1] = f4{v[4], v[5], v[6], v[7]};
      } else {
        Eight o;
#pragma unroll
        for (int k = 0; k < 8; ++k) o.v[k] = from_f32<TX>(v[k]);
        *reinterpret_cast<Eight*>(static_cast<TX*>(d.out) + outer_at(a, d, ch.e, r + wave, c0)) = o;
      }
    }
  }
}

// m in fp32, multiplied as it is; TX: the type of the result.
template <class TX, int RF, bool FEW>
__device__ __forceinline__ void outer_32(const AdaptOuter& a, const AdaptOuter::Part& d, const AdaptChunk& ch, uint64_t mine,
                                         int c_group, int r0, float* s_sum) {
  constexpr int U = 4;  // steps of four positions
  int w0, w1;
  wave_part(ch, w0, w1);
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, c0 = c_group + 4 * i;
  const bool in = c0 < d.C;
  f4 acc[RF][4], mn[U];
  float vn[RF][U];
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[f][k] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  int row[U];
  const float* m_col = static_cast<const float*>(d.m) + min(c0, d.C - 4);
  auto rows_of = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = max(min(p + 4 * u + g, w1 - 1), 0);
      row[u] = !FEW && d.order ? d.order[t] : t;
    }
  };
  auto fetch = [&](int p) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = p + 4 * u + g;
      const bool own = t < w1 && (!FEW || (mine >> t & 1));
      if constexpr (FEW) mn[u] = f4{0.0f, 0.0f, 0.0f, 0.0f};
      if (!FEW || own) {  // positions behind the part: its last one's row, times 0
        const float* q = m_col + (size_t)row[u] * d.ldm;
        if (d.vec_m) mn[u] = *reinterpret_cast<const f4*>(q);
        else mn[u] = f4{q[0], q[1], q[2], q[3]};
      }
#pragma unroll
      for (int f = 0; f < RF; ++f) {
        const float v = d.v[(size_t)max(min(t, w1 - 1), 0) * a.R + min(r0 + 16 * f + i, a.R - 1)];
        vn[f][u] = own ? v : 0.0f;
      }
    }
  };
  rows_of(w0);
  fetch(w0);
  rows_of(w0 + 4 * U);
  for (int p = w0; p < w1; p += 4 * U) {
    f4 m[U];
    float v[RF][U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      m[u] = mn[u];
#pragma unroll
      for (int f = 0; f < RF; ++f) v[f][u] = vn[f][u];
    }
    fetch(p + 4 * U);
    rows_of(p + 8 * U);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < RF; ++f)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[f][k] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[f][u], m[u][k], acc[f][k], 0, 0, 0);
  }
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int f = 0; f < RF; ++f)
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) s_sum[(((wave * RF + f) * 4 + k) * 4 + j) * 64 + lane] = acc[f][k][j];
  __syncthreads();
  auto total = [&](int f, int k, int j) __attribute__((always_inline)) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) v += s_sum[(((w * RF + f) * 4 + k) * 4 + j) * 64 + lane];
    return v;
  };
  if (!in) return;
#pragma unroll
  for (int f = 0; f < RF; ++f) {
    const int r = r0 + 16 * f + 4 * g;
    if (r >= a.R) continue;
    const bool rows = ch.slot < 0 && d.rows;  // four rows of a column, or four columns of a row
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = rows ? total(f, wave, k) : total(f, k, wave);
    if (ch.slot >= 0) {
      *reinterpret_cast<f4*>(d.part + ((size_t)ch.slot * a.R + r + wave) * d.C + c0) = f4{v[0], v[1], v[2], v[3]};
    } else {
      Four<TX> o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o.v[k] = from_f32<TX>(v[k]);
      const size_t at = rows ? outer_at(a, d, ch.e, r, c0 + wave) : outer_at(a, d, ch.e, r + wave, c0);
      *reinterpret_cast<Four<TX>*>(static_cast<TX*>(d.out) + at) = o;
    }
  }
}

// columns of a workgroup
template <class TX>
constexpr int outer_cols(bool f32) {
  return f32 || std::is_same<TX, float>::value ? 64 : 128;
}
template <class TX, int RF, bool FEW>
__device__ __forceinline__ void outer_run(const AdaptOuter& a, const AdaptOuter::Part& d, const AdaptChunk& ch, uint64_t mine,
                                          int c, int r0, float* s_sum) {
  if constexpr (std::is_same<TX, float>::value) {
    outer_32<TX, RF, FEW>(a, d, ch, mine, c, r0, s_sum);
  } else if (d.f32) {
    outer_32<TX, RF, FEW>(a, d, ch, mine, c, r0, s_sum);
  } else {
    outer_16<TX, RF, FEW>(a, d, ch, mine, c, r0, s_sum);
  }
}

// Workgroups in x: the columns of the first gradient, then of the second. In y: runs of positions, then adapters, whose
// gradients are zeros where they have no tokens.
template <class TX, int RF, bool FEW>
__global__ __launch_bounds__(256, 2) void k_adapt_outer(AdaptOuter a, int x0, int runs) {
  __shared__ __align__(16) float s_sum[4 * RF * 16 * outer_cols<TX>(false)];
  const bool second = (int)blockIdx.x >= x0;
  const AdaptOuter::Part& d = a.part[second];
  const int cols = outer_cols<TX>(d.f32), c = (blockIdx.x - (second ? x0 : 0)) * cols, r0 = blockIdx.z * 16 * RF;
  if constexpr (FEW) {  // an adapter each; without tokens its sums are zeros
    const int lane = threadIdx.x & 63;
    const uint64_t mine = __ballot(lane < a.T && (a.ids ? a.ids[min(lane, a.T - 1)] : 0) == (int)blockIdx.y);
    const AdaptChunk ch{(int)blockIdx.y, 0, mine ? a.T : 0, -1};
    outer_run<TX, RF, true>(a, d, ch, mine, c, r0, s_sum);
    return;
  }
  if ((int)blockIdx.y >= runs) {
    const int e = blockIdx.y - runs;
    if (a.order.offsets[e + 1] != a.order.offsets[e]) return;
    const int rows = min(16 * RF, a.R - r0);
    for (int k = threadIdx.x; k < rows * cols; k += 256) {
      const int r = d.rows ? k % rows : k / cols, cc = c + (d.rows ? k / rows : k % cols);
      if (cc < d.C) static_cast<TX*>(d.out)[outer_at(a, d, e, r0 + r, cc)] = from_f32<TX>(0.0f);
    }
    return;
  }
  if ((int)blockIdx.y >= *a.order.n_chunks) return;
  const AdaptChunk ch = a.order.chunks[blockIdx.y];
  outer_run<TX, RF, false>(a, d, ch, 0, c, r0, s_sum);
}

// Adapters of several runs: their partial sums in ascending order.
template <class TX>
__global__ __launch_bounds__(256) void k_adapt_join(AdaptOuter a, int x0, int len) {
  const bool second = (int)blockIdx.x >= x0;
  const AdaptOuter::Part& d = a.part[second];
  const int c = (blockIdx.x - (second ? x0 : 0)) * 256 + threadIdx.x, r0 = blockIdx.z * 8, e = blockIdx.y;
  const int n = (a.order.offsets[e + 1] - a.order.offsets[e] + len - 1) / len;
  if (n < 2 || c >= d.C) return;
  float v[8] = {};
  const float* part = d.part + ((size_t)a.order.slot0[e] * a.R + r0) * d.C + c;
#pragma unroll 2
  for (int k = 0; k < n; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += part[((size_t)k * a.R + j) * d.C];
  TX o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = from_f32<TX>(v[j]);
  TX* to = static_cast<TX*>(d.out) + outer_at(a, d, e, r0, c);
  if (d.rows) {
#pragma unroll
    for (int j = 0; j < (int)(sizeof(TX) / 2); ++j) reinterpret_cast<u4v*>(to)[j] = reinterpret_cast<const u4v*>(o)[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) to[(size_t)j * d.C] = o[j];
  }
}

// Tiles of 32 x 32 of the first matrix, then of the second.
template <class V>
__global__ __launch_bounds__(256) void k_adapt_transpose(AdaptTranspose a, int x0) {
  __shared__ V s[32][33];
  const int e = blockIdx.y;
  if (a.offsets[e + 1] == a.offsets[e]) return;
  const bool second = (int)blockIdx.x >= x0;
  const AdaptTranspose::Part& d = a.part[second];
  const int k0 = blockIdx.x - (second ? x0 : 0), across = (d.Q + 31) / 32;
  const int q0 = k0 % across * 32, m0 = k0 / across * 32, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const size_t base = (size_t)e * d.M * d.Q;
  const V* in = static_cast<const V*>(d.in) + base;
  V* out = static_cast<V*>(d.out) + base;
#pragma unroll
  for (int k = ty; k < 32; k += 8)
    if (m0 + k < d.M && q0 + tx < d.Q) s[k][tx] = in[(size_t)(m0 + k) * d.Q + q0 + tx];
  __syncthreads();
#pragma unroll
  for (int k = ty; k < 32; k += 8)
    if (q0 + k < d.Q && m0 + tx < d.M) out[(size_t)(q0 + k) * d.M + m0 + tx] = s[tx][k];
}

template <class TX>
void down_launch(const AdaptDown& a, hipStream_t st) {
  if (a.few) {
    k_adapt_dot<TX><<<dim3(a.T, a.R / 4, a.parts), 256, 0, st>>>(a);
    return;
  }
  const int groups = a.runs ? (int)adapt_max_runs(a.T, a.n_ad) : (a.T + 15) / 16;
  if (a.R <= 16 || (a.T + 15) / 16 * ((a.R + 31) / 32) < 256)
    k_adapt_down<TX, 1><<<dim3(groups, (a.R + 15) / 16, a.parts), 64 * kDownWaves, 0, st>>>(a);
  else
    k_adapt_down<TX, 2><<<dim3(groups, (a.R + 31) / 32, a.parts), 64 * kDownWaves, 0, st>>>(a);
}
template <class TX>
void outer_launch(const AdaptOuter& a, hipStream_t st) {
  const int len = adapt_chunk_len(a.T);
  auto cols = [&](int k, int w) { return a.part[k].out ? (a.part[k].C + w - 1) / w : 0; };
  const int x0 = cols(0, outer_cols<TX>(a.part[0].f32)), x = x0 + cols(1, outer_cols<TX>(a.part[1].f32));
  if (!a.order.order) {
    if (a.R <= 16) k_adapt_outer<TX, 1, true><<<dim3(x, a.n_ad), 256, 0, st>>>(a, x0, 0);
    else k_adapt_outer<TX, 2, true><<<dim3(x, a.n_ad, (a.R + 31) / 32), 256, 0, st>>>(a, x0, 0);
    return;
  }
  const int runs = (int)adapt_max_chunks(a.T, a.n_ad);
  if (a.R <= 16) k_adapt_outer<TX, 1, false><<<dim3(x, runs + a.n_ad), 256, 0, st>>>(a, x0, runs);
  else k_adapt_outer<TX, 2, false><<<dim3(x, runs + a.n_ad, (a.R + 31) / 32), 256, 0, st>>>(a, x0, runs);
  if (a.T > len)
    k_adapt_join<TX><<<dim3(cols(0, 256) + cols(1, 256), a.n_ad, a.R / 8), 256, 0, st>>>(a, cols(0, 256), len);
}

}  // namespace

hipError_t launch_adapt_order(const int32_t* ids, int T, int n_ad, const AdaptOrder& out, hipStream_t st) {
  k_adapt_order<<<1, 64 * kOrderWaves, 0, st>>>(ids, T, n_ad, out, out.offsets ? adapt_chunk_len(T) : 0);
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
hipError_t launch_adapt_transpose(const AdaptTranspose& a, int elem, hipStream_t st) {
  auto tiles = [&](int k) { return a.part[k].out ? (a.part[k].Q + 31) / 32 * ((a.part[k].M + 31) / 32) : 0; };
  const dim3 grid(tiles(0) + tiles(1), a.n_ad);
  if (elem == 4) k_adapt_transpose<uint32_t><<<grid, 256, 0, st>>>(a, tiles(0));
  else k_adapt_transpose<uint16_t><<<grid, 256, 0, st>>>(a, tiles(0));
  return hipGetLastError();
}

}  // namespace moe
