// k_route.hip — routing from given logits (softmax or sigmoid scores, selection bias, groups, top-K, load
// statistics), its gradient, and the gradient of the routing weights from the experts' outputs.
//
// One wavefront works on one token: lane l holds the NE consecutive experts l*NE .. l*NE + NE-1, so the lowest
// lane and, in it, the lowest register that hold a value hold its lowest expert, which is the tie rule.
#include <algorithm>
#include <type_traits>

#include "moe_float.h"
#include "moe_ops.h"

namespace moe {

namespace {

constexpr int kWaves = 4;  // wavefronts per workgroup

// ------------------------------------------------------------ wavefront reductions
// A row of 16 lanes by quad permutes and mirrors, then the rows by the two row broadcasts; lane 63 holds the
// result of all 64 lanes and readlane makes it uniform. No LDS round trip.
// Every lane of these patterns has a source, so the move can be part of the instruction that uses it.
template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
// the same into the rows of the mask only; the others get `old`, which has no effect on the reduction
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_rows(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_max_i(int v) {
  v = max(v, dpp_i<0xB1>(v));   // quad_perm [1,0,3,2]
  v = max(v, dpp_i<0x4E>(v));   // quad_perm [2,3,0,1]
  v = max(v, dpp_i<0x141>(v));  // row_half_mirror
  v = max(v, dpp_i<0x140>(v));  // row_mirror
  v = max(v, dpp_rows<0x142, 0xA>(INT32_MIN, v));  // row_bcast15 into rows 1 and 3
  v = max(v, dpp_rows<0x143, 0xC>(INT32_MIN, v));  // row_bcast31 into rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, dpp_i<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add_rows(float v) {
  return v + __builtin_bit_cast(float, dpp_rows<CTRL, ROWS>(0, __builtin_bit_cast(int, v)));
}
__device__ __forceinline__ float readlane_f(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
// fixed order: pairs, quads, halves, rows
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  v = dpp_add<0x140>(v);
  v = dpp_add_rows<0x142, 0xA>(v);
  v = dpp_add_rows<0x143, 0xC>(v);
  return readlane_f(v, 63);
}
__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// Order-preserving signed integer of a float that is not NaN (-0 has to be made +0 by the caller).
__device__ __forceinline__ int okey(float f) {
  const int b = __float_as_int(f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float unkey(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }
constexpr int kDead = INT32_MIN;  // below the key of every number (-inf is 0x807FFFFF)

// ------------------------------------------------------------ one token's row
// Lane's NE logits as fp32 (+inf becomes the largest fp32) and, in the result, a bit per live one. vec: the lane's
// run is whole, in one vector load.
template <int NE, class TZ>
struct alignas(NE * sizeof(TZ) < 16 ? NE * sizeof(TZ) : 16) Run {
  TZ v[NE];
};
template <int NE, class TZ>
__device__ __forceinline__ uint32_t load_row(const TZ* row, int E, bool vec, int lane, float (&z)[NE]) {
  const int e0 = lane * NE;
  float f[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) f[i] = kNegInf;
  if (vec) {  // E is a multiple of NE
    if (e0 < E) {
      const Run<NE, TZ> r = *reinterpret_cast<const Run<NE, TZ>*>(row + e0);
#pragma unroll
      for (int i = 0; i < NE; ++i) f[i] = to_f32<TZ>(r.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (e0 + i < E) f[i] = to_f32<TZ>(row[e0 + i]);
  }
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const bool on = f[i] > lowest<TZ>();
    z[i] = on ? __builtin_amdgcn_fmed3f(f[i], -3.402823466e38f, 3.402823466e38f) + 0.0f : kNegInf;
    live |= on ? 1u << i : 0u;
  }
  return live;
}

template <int NE>
__device__ __forceinline__ float row_max(const float (&z)[NE]) {
  int m = kDead;
#pragma unroll
  for (int i = 0; i < NE; ++i) m = max(m, okey(z[i]));
  return unkey(wave_max_i(m));
}

// ------------------------------------------------------------ forward
struct RouteArgs {
  const void* logits;
  int64_t ld;
  int32_t T, E, G, KG, K;
  int32_t group_max, renorm, vec;
  int32_t glog;  // log2 of the lanes of a group, -1 where groups are not whole lanes or not a power of two of them
  float scale;
  const float* bias;
  const uint8_t* valid;
  int32_t* ids;
  float* w;
  int32_t* load;   // [E], or null
  float* imp;      // [E], or null
  int32_t* pload;  // [blocks][E] partial counts, and
  float* pimp;     // [blocks][E] partial sums of the workgroups
};

// Orders LDS writes of some lanes of a wavefront before later LDS reads of others (and those before later writes).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// lanes of the mask below this one, and c
__device__ __forceinline__ int lanes_below(uint64_t m, int c) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, c));
}

// (a, b) two largest of one set, (c, d) of another -> of both
__device__ __forceinline__ void merge_top2(int& a, int& b, int c, int d) {
  b = max(max(b, d), min(a, c));
  a = max(a, c);
}
template <int CTRL>
__device__ __forceinline__ void merge_top2_dpp(int& a, int& b) {
  merge_top2(a, b, dpp_i<CTRL>(a), dpp_i<CTRL>(b));
}

// Group limiting: which of the lane's experts stay. g[i] is the value that the groups are scored by (kDead where
// masked). The score is the sum of the two largest of a group (of the one, where it has one) or the largest; the KG
// best groups stay, the lower index first on equal scores. *near is set where the last kept and the first dropped
// group lie within thr + 1e-6 of the sum of their addends' magnitudes: adding a score to its bias loses up to 2^-24 of
// either's result, which the sum of two opposite ones need not show. A difference that is no number is near, too.
// glog >= 0: a group is 2^glog whole lanes, its two largest are merged across them in registers; else its run is
// scanned in LDS by one lane. 32,768 tokens x 256 experts in 8 groups: 35.4 us with the merge, 44.5 with the scan; one
// token 4.2 and 5.5.
template <int NE>
__device__ __forceinline__ uint32_t keep_groups(const int (&g)[NE], int E, int G, int KG, int glog, bool gmax, int lane,
                                                int* s_row, float thr, bool* near) {
  int a = kDead, b = kDead, mine, step;
  if (glog >= 0) {
#pragma unroll
    for (int i = 0; i < NE; ++i) merge_top2(a, b, g[i], kDead);
    if (glog >= 1) merge_top2_dpp<0xB1>(a, b);   // quad_perm [1,0,3,2]
    if (glog >= 2) merge_top2_dpp<0x4E>(a, b);   // quad_perm [2,3,0,1]
    if (glog >= 3) merge_top2_dpp<0x141>(a, b);  // row_half_mirror
    if (glog >= 4) merge_top2_dpp<0x140>(a, b);  // row_mirror
    if (glog >= 5) merge_top2(a, b, __shfl_xor(a, 16), __shfl_xor(b, 16));
    if (glog >= 6) merge_top2(a, b, __shfl_xor(a, 32), __shfl_xor(b, 32));
    mine = lane >> glog;
    step = 1 << glog;
  } else {
    const int n = E / G;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane * NE + i < E) s_row[lane * NE + i] = g[i];
    wave_sync();
    if (lane < G)
      for (int j = 0; j < n; ++j) merge_top2(a, b, s_row[lane * n + j], kDead);
    wave_sync();
    mine = lane;
    step = 1;
  }
  const bool is = mine < G;
  const bool one = gmax || b == kDead;
  const int score = !is ? kDead : one ? a : okey(__fadd_rn(unkey(a), unkey(b)) + 0.0f);
  const float size = fabsf(unkey(a)) + (one ? 0.0f : fabsf(unkey(b)));
  int rank = 0;
  if (G <= 8) {  // all pairs at once: lane 8a + b compares group b with group a
    const int pa = __shfl(score, (lane >> 3) * step), pb = __shfl(score, (lane & 7) * step);
    const uint64_t ahead = __ballot((lane & 7) < G && pb + ((lane & 7) < lane >> 3 ? 1 : 0) > pa);
    rank = __popc((uint32_t)(ahead >> (mine & 7) * 8) & 0xFFu);
  } else {
    for (int h = 0; h < G; ++h) {
      const int o = __builtin_amdgcn_readlane(score, h * step);
      rank += o + (h < mine ? 1 : 0) > score;  // keys of numbers stay below INT32_MAX
    }
  }
  const bool kept = is && rank < KG && score != kDead;
  const uint64_t m = __ballot(kept), last = __ballot(is && rank == KG - 1), next = __ballot(is && rank == KG);
  *near = false;
  if (next) {  // the last group kept and the best one dropped
    const int lp = __ffsll((unsigned long long)last) - 1, lq = __ffsll((unsigned long long)next) - 1;
    const int kp = __builtin_amdgcn_readlane(score, lp), kq = __builtin_amdgcn_readlane(score, lq);
    if (kp != kDead && kq != kDead)
      *near = !(unkey(kp) - unkey(kq) > thr + 1e-6f * (readlane_f(size, lp) + readlane_f(size, lq)));
  }
  uint32_t r = 0;
  if (glog >= 0) {
    r = kept ? (1u << NE) - 1 : 0;
  } else {
    const int n = E / G;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane * NE + i < E && (m >> ((lane * NE + i) / n) & 1)) r |= 1u << i;
  }
  return r;
}

// The K largest keys of the wavefront (all, where there are fewer; the lower index first on equal keys), in no order:
// their number, and lane j < number holds the key and the expert of one of them, in *key and *id. *next is the
// largest key left out (kDead: none).
// The K-th largest is found by bisection between keys: a step is NE comparisons whose ballots are counted in scalar
// registers, and about ten steps separate the K-th from the next; K rounds of a largest key took 20 vector
// instructions each and 6 dependent lane moves.
template <int NE>
__device__ __forceinline__ int top_keys(const int (&k)[NE], int K, int lane, int* scratch, int* key, int* id, int* next) {
  int lm = k[0];
#pragma unroll
  for (int i = 1; i < NE; ++i) lm = max(lm, k[i]);
  const int top = wave_max_i(lm);
  // every lane with a live key has one that is at least the smallest of their largest ones
  const uint64_t lanes = __ballot(lm != kDead);
  const int base = __popcll(lanes) >= K ? -wave_max_i(lm != kDead ? -lm : kDead) : kDead + 1;
  auto count = [&](int v) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) c += __popcll(__ballot(k[i] >= v));
    return c;
  };
  int lo = base, n_lo = count(base), hi = top, n_hi = 0;  // count(lo) >= K > count(hi + 1), where there are K
  while (n_lo > K && lo != hi) {  // the smallest v > lo with count(v) <= K lies in (lo, hi + 1]
    const int mid = (int)((uint32_t)lo + (((uint32_t)hi - (uint32_t)lo + 1u) >> 1));
    const int c = count(mid);
    const bool up = c >= K;
    lo = up ? mid : lo;
    n_lo = up ? c : n_lo;
    hi = up ? hi : mid - 1;
    n_hi = up ? n_hi : c;
  }
  int kk[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) kk[i] = k[i];
  int rest = kDead;
  if (n_lo > K) {  // more than K keys are at least lo, n_hi of them above it: the first K - n_hi that equal lo fill up
    int before = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) before += lanes_below(__ballot(k[i] == lo), 0);
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (k[i] == lo && before++ >= K - n_hi) kk[i] = kDead;
    rest = lo;
  }
  int at = 0;
  uint2* slot = reinterpret_cast<uint2*>(scratch);
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const bool on = kk[i] >= lo;
    const uint64_t m = __ballot(on);
    if (on) slot[lanes_below(m, at)] = make_uint2((uint32_t)kk[i], (uint32_t)(lane * NE + i));
    at += __popcll(m);
    rest = max(rest, on ? kDead : kk[i]);
  }
  wave_sync();
  const uint2 mine = lane < at ? slot[lane] : make_uint2((uint32_t)kDead, 0xFFFFFFFFu);
  wave_sync();
  *key = (int)mine.x;
  *id = (int)mine.y;
  *next = wave_max_i(rest);
  return at;
}

// Rank of the lane's key among the first n lanes' (larger first, the lower id first on equal keys).
__device__ __forceinline__ int rank_of(int key, int id, int n, int lane) {
  int rank = 0;
  if (n <= 8) {  // all pairs at once: lane 8a + b compares key b with key a
    const int ka = __shfl(key, lane >> 3), kb = __shfl(key, lane & 7), ia = __shfl(id, lane >> 3), ib = __shfl(id, lane & 7);
    const uint64_t ahead = __ballot((lane & 7) < n && (kb > ka || (kb == ka && ib < ia)));
    rank = __popc((uint32_t)(ahead >> (lane & 7) * 8) & 0xFFu);
  } else {
    for (int j = 0; j < n; ++j) {
      const int ok = __builtin_amdgcn_readlane(key, j), oi = __builtin_amdgcn_readlane(id, j);
      rank += ok > key || (ok == key && oi < id);
    }
  }
  return rank;
}

// e^x (x <= 0) and sigmoid for comparing scores: the argument of 2^x is rounded once, which for the scores, 1 / (1 +
// e^-|z|) or e^(z - max) / sum, is below 4e-8 of the largest, however large |z| is.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
__device__ __forceinline__ float sigmoid_fast(float z) {
  const float a = exp_fast(-fabsf(z)), d = __builtin_amdgcn_rcpf(1.0f + a);
  return z >= 0.0f ? d : a * d;
}

// Wavefronts of k_route that a SIMD holds at a time, by experts a lane.
constexpr int resident_waves(int ne) { return ne <= 4 ? 6 : ne == 8 ? 4 : 2; }

// The definition compares fl32(score) + bias, the score taken in 64 bits, so that every implementation chooses the
// same experts. Taking 256 exponentials a token in 64 bits would be most of the work; so the choice is made with 32-bit
// scores, and a token where two neighbours in the order (or two groups) lie closer than twice the error of those (see
// thr) is set aside and done once more with the definition's: 2 tokens in 1,000 of 256 biased sigmoid scores.
// Bound by instruction issue, not by its bytes: 340 vector and 270 scalar instructions a token of 256 experts in 8
// groups with bias and statistics, the former 73% of the SIMDs' cycles, 35.8 us for 32,768 of them (36 MB); one token
// 3.9 us, 192 softmax ones of 128 5.0. The six wavefronts a SIMD of 129 to 256 experts cost 2 to 6 spilled vector
// registers with softmax or statistics.
template <int NE, class TZ, bool SOFTMAX, bool STATS, int WV>
__global__ __launch_bounds__(64 * WV, resident_waves(NE)) void k_route(RouteArgs a) {
  __shared__ __align__(8) int s_row[WV][64 * NE];  // a wavefront's scratch
  __shared__ int s_load[STATS ? 64 * NE : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, K = a.K;
  int* scratch = s_row[wave];
  float bias[NE], imp[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    bias[i] = a.bias && lane * NE + i < E ? a.bias[lane * NE + i] : 0.0f;
    imp[i] = 0.0f;
  }
  if (STATS) {
    for (int e = threadIdx.x; e < 64 * NE; e += 64 * WV) s_load[e] = 0;
    __syncthreads();
  }
  const bool by_sum = a.G > 1 && !a.group_max;
  const bool scored = a.bias || by_sum;  // the choice compares scores, not logits

  // one token; true where it has to be done with exact scores instead (then nothing is written)
  auto token = [&](int t, auto exact_) __attribute__((always_inline)) -> bool {
    constexpr bool EXACT = decltype(exact_)::value;
    const TZ* row = static_cast<const TZ*>(a.logits) + (size_t)t * a.ld;
    if (a.valid && a.valid[t] == 0) {
      if (lane < K) {
        a.ids[(size_t)t * K + lane] = -1;
        a.w[(size_t)t * K + lane] = 0.0f;
      }
      return false;
    }
    float z[NE], s[NE];
    const uint32_t live = load_row<NE, TZ>(row, E, a.vec, lane, z);
    float m = 0.0f, rs = 0.0f;  // softmax: largest logit (-inf: nothing to choose from), 1 / sum
    if constexpr (SOFTMAX) {
      m = row_max<NE>(z);
      if (scored || STATS || !a.renorm) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          s[i] = live >> i & 1 ? exp_fast(z[i] - m) : 0.0f;
          sum += s[i];
        }
        rs = safe_rcp(wave_sum(sum));
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] *= rs;
      }
    } else if (scored || STATS) {
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = live >> i & 1 ? sigmoid_fast(z[i]) : 0.0f;
    }
    if constexpr (STATS && !EXACT) {
      if constexpr (SOFTMAX) {
#pragma unroll
        for (int i = 0; i < NE; ++i) imp[i] += s[i];
      } else {
        float q[NE], sum = 0.0f, zm = z[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) zm = fmaxf(zm, z[i]);
        const bool low = __ballot(zm >= -40.0f) == 0;  // the sum would underflow: relative to the largest logit
        const float ref = low ? row_max<NE>(z) : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          q[i] = s[i];
          if (low) q[i] = live >> i & 1 ? sigmoid_rel(z[i], ref) : 0.0f;
          sum += q[i];
        }
        const float r = safe_rcp(wave_sum(sum));
#pragma unroll
        for (int i = 0; i < NE; ++i) imp[i] = fmaf(q[i], r, imp[i]);
      }
    }
    if constexpr (EXACT) {  // through LDS, one expert of the lane at a time: rare, and it should not cost registers
      float* f = reinterpret_cast<float*>(scratch) + lane * NE;
#pragma unroll
      for (int i = 0; i < NE; ++i) f[i] = z[i];
      double sum = 0.0;
      if (SOFTMAX) {
#pragma unroll 1
        for (int i = 0; i < NE; ++i)
          if (f[i] > kNegInf) sum += exp((double)f[i] - (double)m);
        sum = wave_sum_d(sum);
      }
#pragma unroll 1
      for (int i = 0; i < NE; ++i) {
        const double zi = f[i];
        f[i] = !(f[i] > kNegInf) ? 0.0f
                                 : (float)(SOFTMAX ? exp(zi - (double)m) / sum : 1.0 / (1.0 + exp(-zi)));
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) s[i] = f[i];
      wave_sync();
    }
    // Twice the error of a 32-bit score. Sigmoid: e^-|z| 2.1e-7, the sum, reciprocal and product 2.4e-7, weighted by at
    // most 1/4 and 1: below 3e-7, and 6e-8 for rounding the 64-bit score. Softmax: the sum of up to 1024 terms
    // (21 roundings along a path) 1.3e-6, the exponential, reciprocal and product 4e-7, of the largest score rs.
    const float thr = SOFTMAX ? 4.5e-6f * rs + 1e-7f : 1.0e-6f;
    int key[NE];
    bool near = false;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float c = a.bias ? __fadd_rn(s[i], bias[i]) + 0.0f : z[i];
      key[i] = (live >> i & 1) && c > kNegInf ? okey(c) : kDead;
    }
    if (a.G > 1) {
      int gk[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) gk[i] = by_sum && !a.bias ? (live >> i & 1 ? okey(s[i]) : kDead) : key[i];
      const uint32_t keep = keep_groups<NE>(gk, E, a.G, a.KG, a.glog, a.group_max, lane, scratch, 2.0f * thr, &near);
#pragma unroll
      for (int i = 0; i < NE; ++i) key[i] = keep >> i & 1 ? key[i] : kDead;
    }
    int my_key, my_id, next;
    const int n_sel = top_keys<NE>(key, K, lane, scratch, &my_key, &my_id, &next);
    const bool on = lane < n_sel;
    float my_z = kNegInf;  // read again: the logit of a chosen expert
    if (on) my_z = fminf(to_f32<TZ>(row[my_id]), 3.402823466e38f) + 0.0f;
    const int rank = rank_of(my_key, my_id, n_sel, lane);
    if (!EXACT && scored) {
      if (a.bias) {  // the chosen in order, and the best one left out
        if (on) scratch[rank] = my_key;
        if (lane == 0) scratch[n_sel] = next;
        wave_sync();
        const int nk = on ? scratch[rank + 1] : kDead;
        wave_sync();
        const float p = unkey(my_key), gap = p - unkey(nk);
        // the rounding of the two additions is below 1e-6 of the values
        near |= __ballot(on && nk != kDead && gap <= thr + 1e-6f * (fabsf(p) + gap)) != 0;
      }
      if (near) return true;
    }
    float r;
    if (a.renorm) {
      float q;
      if (!SOFTMAX && __ballot(on && my_z < -40.0f) == 0) {
        float miss;
        sigmoid2(my_z, q, miss);
        q = on ? q : 0.0f;
      } else {
        const float ref = unkey(wave_max_i(on ? okey(my_z) : kDead));
        q = !on ? 0.0f : SOFTMAX ? exp_neg(my_z - ref) : sigmoid_rel(my_z, fminf(ref, 0.0f));
      }
      r = q * safe_rcp(wave_sum(q));
    } else if (SOFTMAX) {
      r = exp_neg(my_z - m) * rs;
    } else {
      float miss;
      sigmoid2(my_z, r, miss);
    }
    if (lane < K) {  // the chosen by their rank, the empty slots behind them
      const int k = on ? rank : lane;
      a.ids[(size_t)t * K + k] = on ? my_id : -1;
      a.w[(size_t)t * K + k] = on ? r * a.scale : 0.0f;
      if (STATS && on) atomicAdd(&s_load[my_id], 1);
    }
    return false;
  };

  const int step = gridDim.x * WV;
  for (int t0 = blockIdx.x * WV + wave; t0 < a.T; t0 += 64 * step) {
    uint64_t again = 0;
    for (int i = 0; i < 64 && t0 + i * step < a.T; ++i)
      if (token(t0 + i * step, std::false_type{})) again |= 1ull << i;
    while (again) {
      const int i = __ffsll((unsigned long long)again) - 1;
      again &= again - 1;
      token(t0 + i * step, std::true_type{});
    }
  }
  if (STATS) {
    float* s_imp = reinterpret_cast<float*>(s_row[0]);  // [WV][64 * NE]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NE; ++i) s_imp[wave * 64 * NE + lane * NE + i] = imp[i];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 64 * WV) {
      float v = s_imp[e];
#pragma unroll
      for (int w = 1; w < WV; ++w) v += s_imp[w * 64 * NE + e];
      a.pload[(size_t)blockIdx.x * E + e] = s_load[e];
      a.pimp[(size_t)blockIdx.x * E + e] = v;
    }
  }
}

// Sums the workgroups' partial statistics in a fixed order: 16 experts a workgroup, 64 lanes of rows each.
__global__ __launch_bounds__(1024) void k_route_stats(const int32_t* __restrict__ pload, const float* __restrict__ pimp,
                                                      int blocks, int E, int32_t* __restrict__ load,
                                                      float* __restrict__ imp) {
  __shared__ int s_l[1024];
  __shared__ double s_i[1024];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
  int l = 0;
  double v = 0.0;
  if (e < E) {
#pragma unroll 4
    for (int b = r; b < blocks; b += 64) {
      l += pload[(size_t)b * E + e];
      v += (double)pimp[(size_t)b * E + e];
    }
  }
  s_l[threadIdx.x] = l;
  s_i[threadIdx.x] = v;
  for (int h = 512; h >= 16; h >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < h) {
      s_l[threadIdx.x] += s_l[threadIdx.x + h];
      s_i[threadIdx.x] += s_i[threadIdx.x + h];
    }
  }
  if (r == 0 && e < E) {
    if (load) load[e] = s_l[threadIdx.x];
    if (imp) imp[e] = (float)s_i[threadIdx.x];
  }
}

// ------------------------------------------------------------ backward
// With renormalised weights w_k = scale * r_k, r = s / (sum of the chosen s): dz_k = r_k (u_k - sum_j r_j u_j) m_k, where
// u = scale * dw and m = 1 for softmax scores (their sum cancels), 1 - s for sigmoid ones; without, dz_k = s_k (1 - s_k)
// u_k, or p_e (u_e - sum_j p_j u_j) over all experts. Importance p = s / (sum of s): p_e (g_e - sum_f p_f g_f) m_e.
// One wavefront a token; a slot's part goes through LDS to the lane that holds its expert, and a row is read and written
// once. 32,768 x 256 sigmoid with importance: 18.8 us for 69 MB (10.8 at 6.4 TB/s), bound by instruction issue: 187
// vector instructions a token, 80% of the SIMDs' cycles; 10.5 us without importance, softmax with it 15.7; 381 x 128
// softmax 3.2.
struct RouteGradArgs {
  const void* logits;
  int64_t ld, ld_d;
  int32_t T, E, K, renorm, vec, vec_d;
  float scale;
  const uint8_t* valid;
  const int32_t* ids;
  const float* dw;    // [T][K], or null
  const float* dimp;  // [E], or null
  void* dz;
};

template <int NE, class TZ, bool SOFTMAX>
__global__ __launch_bounds__(64 * kWaves) void k_route_grad(RouteGradArgs a) {
  __shared__ float s_add[kWaves][64 * NE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = a.E, K = a.K;
  float* add = s_add[wave];
  float dimp[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) dimp[i] = a.dimp && lane * NE + i < E ? a.dimp[lane * NE + i] : 0.0f;
  const bool dense = a.dimp || (SOFTMAX && !a.renorm && a.dw);
  for (int t = blockIdx.x * kWaves + wave; t < a.T; t += gridDim.x * kWaves) {
    const TZ* row = static_cast<const TZ*>(a.logits) + (size_t)t * a.ld;
    const bool dead = a.valid && a.valid[t] == 0;
    float out[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) out[i] = 0.0f;
    if (!dead) {
      // slots: lane k holds slot k's expert, its logit and the gradient of its weight
      int id = -1;
      float zk = kNegInf, u = 0.0f;
      if (a.dw && lane < K) {
        id = a.ids[(size_t)t * K + lane];
        if ((unsigned)id < (unsigned)E) {
          const float f = to_f32<TZ>(row[id]);
          if (f > lowest<TZ>()) {
            zk = fminf(f, 3.402823466e38f);
            u = a.dw[(size_t)t * K + lane] * a.scale;
          } else {
            id = -1;
          }
        } else {
          id = -1;
        }
      }
      const bool on = id >= 0;
      float z[NE], p[NE];
      uint32_t live = 0;
      float m = 0.0f, rs = 0.0f;
      if (dense) {
        live = load_row<NE, TZ>(row, E, a.vec, lane, z);
        if (SOFTMAX) {
          m = row_max<NE>(z);
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NE; ++i) {
            p[i] = live >> i & 1 ? exp_neg(z[i] - m) : 0.0f;
            sum += p[i];
          }
          rs = safe_rcp(wave_sum(sum));
#pragma unroll
          for (int i = 0; i < NE; ++i) p[i] *= rs;
        }
      }
      // the slots' own part
      float dk = 0.0f;
      if (a.renorm) {
        float q, miss = 1.0f;
        if (SOFTMAX || __ballot(on && zk < -40.0f)) {
          const float ref = unkey(wave_max_i(on ? okey(zk + 0.0f) : kDead));
          q = !on ? 0.0f : SOFTMAX ? exp_neg(zk - ref) : sigmoid_rel(zk, fminf(ref, 0.0f));
          if (!SOFTMAX) {
            float s;
            sigmoid2(zk, s, miss);
          }
        } else {
          sigmoid2(zk, q, miss);
          q = on ? q : 0.0f;
        }
        const float r = q * safe_rcp(wave_sum(q));
        const float mean = wave_sum(r * u);
        dk = r * (u - mean) * miss;
      } else if (SOFTMAX) {
        // p_k u_k here, and -p_e sum_k p_k u_k over all experts below
        dk = on ? exp_neg(zk - m) * rs * u : 0.0f;
      } else if (on) {
        float s, miss;
        sigmoid2(zk, s, miss);
        dk = u * s * miss;
      }
      if (a.dw) {
#pragma unroll
        for (int i = 0; i < NE; ++i) add[lane * NE + i] = 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (on) atomicAdd(&add[id], dk);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int i = 0; i < NE; ++i) out[i] = add[lane * NE + i];
        __builtin_amdgcn_wave_barrier();
      }
      // A masked expert's entry of dimp may be infinite or NaN (its importance is 0 where a loss may take a logarithm);
      // the token does not depend on it. Seen in dot, which is then taken again without them: 15.7 us for 32,768 x 256
      // softmax, 16.5 with the masked ones left out always.
      bool odd = false;
      if (SOFTMAX && dense) {
        const float own = a.renorm ? 0.0f : dk;
        float dot = own;
#pragma unroll
        for (int i = 0; i < NE; ++i) dot = fmaf(p[i], dimp[i], dot);
        dot = wave_sum(dot);
        odd = !(fabsf(dot) < INFINITY);
        if (odd) {
          dot = own;
#pragma unroll
          for (int i = 0; i < NE; ++i) dot = live >> i & 1 ? fmaf(p[i], dimp[i], dot) : dot;
          dot = wave_sum(dot);
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) out[i] += p[i] * (dimp[i] - dot);
      } else if (dense) {
        float miss[NE], sum = 0.0f, dot = 0.0f, zm = z[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) zm = fmaxf(zm, z[i]);
        const bool low = __ballot(zm >= -40.0f) == 0;  // the sum would underflow: relative to the largest logit
        const float ref = low ? row_max<NE>(z) : 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          sigmoid2(z[i], p[i], miss[i]);
          if (low) p[i] = sigmoid_rel(z[i], ref);
          p[i] = live >> i & 1 ? p[i] : 0.0f;
          sum += p[i];
          dot = fmaf(p[i], dimp[i], dot);
        }
        rs = safe_rcp(wave_sum(sum));
        dot = wave_sum(dot);
        odd = !(fabsf(dot) < INFINITY);
        if (odd) {
          dot = 0.0f;
#pragma unroll
          for (int i = 0; i < NE; ++i) dot = live >> i & 1 ? fmaf(p[i], dimp[i], dot) : dot;
          dot = wave_sum(dot);
        }
        dot *= rs;
#pragma unroll
        for (int i = 0; i < NE; ++i) out[i] += p[i] * rs * (dimp[i] - dot) * miss[i];
      }
      if (odd)
#pragma unroll
        for (int i = 0; i < NE; ++i) out[i] = live >> i & 1 ? out[i] : 0.0f;
    }
    TZ* drow = static_cast<TZ*>(a.dz) + (size_t)t * a.ld_d;
    const int e0 = lane * NE;
    Run<NE, TZ> r;
#pragma unroll
    for (int i = 0; i < NE; ++i) r.v[i] = from_f32<TZ>(out[i]);
    if (a.vec_d) {
      if (e0 < E) *reinterpret_cast<Run<NE, TZ>*>(drow + e0) = r;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (e0 + i < E) drow[e0 + i] = r.v[i];
    }
  }
}

// ------------------------------------------------------------ gradient of the routing weights
// dw[t][k] = sum_h dy[t][h] e_out[t*K + k][h]. Reads every slot's row once: HBM-bound. One wavefront takes one slot,
// eight 16-byte loads of its row in flight (not kept in the caches); the K slots of a token sit next to each other, so
// dy comes from the caches after the first. 2,048 x 8 x 6144: 70.6 us, 6.4 TB/s (80.4 with one load in flight).
constexpr int kSlotLoads = 8;
typedef float f4v __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(256) void k_slot_grad(const float* __restrict__ eout, const int32_t* __restrict__ ids,
                                                   const float* __restrict__ dy, int64_t slots, int K, int H,
                                                   uint32_t id_end, float* __restrict__ dw) {
  const int lane = threadIdx.x & 63;
  const int64_t j = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (j >= slots) return;
  f4v v = {0.0f, 0.0f, 0.0f, 0.0f};
  if ((uint32_t)ids[j] < id_end) {
    const f4v* a = reinterpret_cast<const f4v*>(eout + (size_t)j * H);
    const f4v* b = reinterpret_cast<const f4v*>(dy + (size_t)(j / K) * H);
    const int n = H / 4;
    int h = lane;
    for (; h + 64 * (kSlotLoads - 1) < n; h += 64 * kSlotLoads) {
      f4v x[kSlotLoads], y[kSlotLoads];
#pragma unroll
      for (int i = 0; i < kSlotLoads; ++i) x[i] = __builtin_nontemporal_load(a + h + 64 * i);
#pragma unroll
      for (int i = 0; i < kSlotLoads; ++i) y[i] = b[h + 64 * i];
#pragma unroll
      for (int i = 0; i < kSlotLoads; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = fmaf(x[i][c], y[i][c], v[c]);
    }
    for (; h < n; h += 64) {
      const f4v x = a[h], y = b[h];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = fmaf(x[c], y[c], v[c]);
    }
  }
  const float sum = wave_sum((v[0] + v[1]) + (v[2] + v[3]));
  if (lane == 0) dw[j] = sum;
}

}  // namespace

// ------------------------------------------------------------ launches
constexpr int kSimds = 1024;
// With statistics a workgroup leaves one row of partial sums; from this many tokens on it has 8 wavefronts, so that
// there are at most 768 rows to add up (32,768 x 256: 5.2 us for them, 8.2 for twice as many).
constexpr int kRouteWideT = 2048;
constexpr int kWideWaves = 8;

static int elems_per_lane(int E) { return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16; }

// Workgroups of `waves` wavefronts for T tokens, at most `per_simd` wavefronts on each SIMD: as many as fit at a time,
// so that all end together. 32,768 tokens x 256 experts, with their statistics added up: 43.7 us, 45.4 with 8 wavefronts a
// SIMD, of which 6 fit.
static int route_blocks(int T, int waves, int per_simd) {
  const int need = (T + waves - 1) / waves, most = kSimds * per_simd / waves;
  return need < most ? need : most;
}
static int stats_waves(int T) { return T >= kRouteWideT ? kWideWaves : kWaves; }

// for any number of tokens up to T: a batch just below the wide form leaves the most rows
size_t route_ws_bytes(int E, int T) {
  const int per_simd = resident_waves(elems_per_lane(E));
  const int narrow = route_blocks(T < kRouteWideT ? T : kRouteWideT - 1, kWaves, per_simd);
  const int rows = T < kRouteWideT ? narrow : std::max(narrow, route_blocks(T, kWideWaves, per_simd));
  return (size_t)rows * E * 8;
}

// a lane's run in one vector access: runs are whole, and base and row stride keep the run's alignment
static bool vec_ok(const void* p, int64_t ld, int E, int ne, size_t size) {
  const size_t al = ne * size < 16 ? ne * size : 16;
  return E % ne == 0 && reinterpret_cast<uintptr_t>(p) % al == 0 && (size_t)ld * size % al == 0;
}

template <class F>
static void by_shape(int E, int dtype, bool softmax, F f) {
  auto by_sm = [&](auto ne, auto tz) {
    if (softmax) f(ne, tz, std::true_type{});
    else f(ne, tz, std::false_type{});
  };
  auto by_type = [&](auto ne) {
    if (dtype == MOE_DTYPE_F32) by_sm(ne, float{});
    else if (dtype == MOE_DTYPE_BF16) by_sm(ne, bf16_t{});
    else by_sm(ne, _Float16{});
  };
  switch (elems_per_lane(E)) {
    case 1: by_type(std::integral_constant<int, 1>{}); break;
    case 2: by_type(std::integral_constant<int, 2>{}); break;
    case 4: by_type(std::integral_constant<int, 4>{}); break;
    case 8: by_type(std::integral_constant<int, 8>{}); break;
    default: by_type(std::integral_constant<int, 16>{}); break;
  }
}

static size_t dtype_size(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

hipError_t launch_moe_route(const moe_route_config& c, const void* logits, int dtype, int64_t ld, int T,
                            const float* bias, const uint8_t* valid, int32_t* ids, float* w, int32_t* load, float* imp,
                            void* ws, hipStream_t st) {
  RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.T = T;
  a.E = c.n_experts;
  a.G = c.n_group;
  a.KG = c.topk_group;
  a.K = c.top_k;
  a.group_max = c.group_score == MOE_GROUP_MAX;
  a.renorm = c.renorm != 0;
  a.vec = vec_ok(logits, ld, a.E, elems_per_lane(a.E), dtype_size(dtype));
  a.scale = c.scale;
  a.bias = bias;
  a.valid = valid;
  a.ids = ids;
  a.w = w;
  a.glog = -1;
  const int gl = a.E / a.G / elems_per_lane(a.E);  // lanes of a group
  if (gl * elems_per_lane(a.E) * a.G == a.E && gl > 0 && (gl & (gl - 1)) == 0)
    for (a.glog = 0; (1 << a.glog) < gl;) ++a.glog;
  const bool stats = load || imp;
  const int waves = stats ? stats_waves(T) : kWaves, blocks = route_blocks(T, waves, resident_waves(elems_per_lane(a.E)));
  if (stats) {
    a.pload = static_cast<int32_t*>(ws);
    a.pimp = reinterpret_cast<float*>(a.pload + (size_t)blocks * a.E);
  }
  by_shape(a.E, dtype, c.score == MOE_SCORE_SOFTMAX, [&](auto ne, auto tz, auto sm) {
    constexpr int NE = decltype(ne)::value;
    using TZ = decltype(tz);
    constexpr bool SM = decltype(sm)::value;
    if (!stats) k_route<NE, TZ, SM, false, kWaves><<<blocks, 64 * kWaves, 0, st>>>(a);
    else if (waves == kWaves) k_route<NE, TZ, SM, true, kWaves><<<blocks, 64 * kWaves, 0, st>>>(a);
    else k_route<NE, TZ, SM, true, kWideWaves><<<blocks, 64 * kWideWaves, 0, st>>>(a);
  });
  if (stats) k_route_stats<<<(a.E + 15) / 16, 1024, 0, st>>>(a.pload, a.pimp, blocks, a.E, load, imp);
  return hipGetLastError();
}

hipError_t launch_moe_route_grad(const moe_route_config& c, const void* logits, int dtype, int64_t ld, int T,
                                 const uint8_t* valid, const int32_t* ids, const float* dw, const float* dimp, void* dz,
                                 int64_t ld_d, hipStream_t st) {
  RouteGradArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ld_d = ld_d;
  a.T = T;
  a.E = c.n_experts;
  a.K = c.top_k;
  a.renorm = c.renorm != 0;
  a.vec = vec_ok(logits, ld, a.E, elems_per_lane(a.E), dtype_size(dtype));
  a.vec_d = vec_ok(dz, ld_d, a.E, elems_per_lane(a.E), dtype_size(dtype));
  a.scale = c.scale;
  a.valid = valid;
  a.ids = ids;
  a.dw = dw;
  a.dimp = dimp;
  a.dz = dz;
  by_shape(a.E, dtype, c.score == MOE_SCORE_SOFTMAX, [&](auto ne, auto tz, auto sm) {
    k_route_grad<decltype(ne)::value, decltype(tz), decltype(sm)::value><<<route_blocks(T, kWaves, 8), 64 * kWaves, 0, st>>>(a);
  });
  return hipGetLastError();
}

hipError_t launch_slot_grad(const float* eout, const int32_t* ids, const float* dy, int T, int K, int H, uint32_t id_end,
                            float* dw, hipStream_t st) {
  const int64_t slots = (int64_t)T * K;
  k_slot_grad<<<(unsigned)((slots + 3) / 4), 256, 0, st>>>(eout, ids, dy, slots, K, H, id_end, dw);
  return hipGetLastError();
}

}  // namespace moe
