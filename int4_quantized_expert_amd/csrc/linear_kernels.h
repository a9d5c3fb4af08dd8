// linear_kernels.h — the kernels of y = act(W x + b) + r.
#pragma once

#include "linear_common.h"

namespace moe {

namespace {

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
  const TX* row = static_cast<const TX*>(a.x) + (size_t)(in ? token_of(a, t) : 0) * a.ldx;
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
constexpr size_t tile_x_lds() {  // activations of all groups
  return (size_t)KW * 2 * TT * (std::is_same<TX, float>::value ? 2 : 1) * 4096;
}
template <class TX, int TT, int W, int RW, int KW>
constexpr size_t tile_lds() {
  return std::max<size_t>({tile_x_lds<TX, TT, RW, KW>() + (kTransposed ? (size_t)RW * KW * 512 * W : 0),
                           (size_t)(KW / 2) * RW * 8 * 1024, (size_t)16 * kOutRow * 4});
}

// ------------------------------------------------------------ adapters of a fragment
// Column that the sums' position j of a fragment stands for: transposed int8 codes keep the order of a row's bytes, in
// each eight the even elements and then the odd ones.
template <int W>
__device__ __forceinline__ int column_at(int j) {
  if (!kTransposed || W == 4) return j;
  return (j & ~7) + ((j & 4) ? 2 * (j & 3) + 1 : 2 * (j & 3));
}

// d[f] = what their adapters add to the 32 positions from p0 on and the 32 output rows first[f] + l % 32, in the layout
// and the power of two of the tile's sums; 0 for positions without one. One product for each adapter that the positions
// have, of all 32 of them, whose results are taken by the adapter's own positions only: what another adapter holds,
// infinities and NaN included, stays out of theirs. h has two bf16 parts (2^-17 of its value is lost), a bf16 b one and an
// fp16 b two; the product of the two low parts, up to 2^-16 of a term, is left out. fp32 is multiplied as it is.
template <class TX>
__device__ __forceinline__ void adapter_frags(const LinearArgs& a, int p0, const int (&row)[2], int lane, f16v (&d)[2]) {
  const int r = lane & 31, g = lane >> 5, p = min(p0 + r, a.T - 1);
  const int id = p0 + r < a.T ? adapter_of(a, p) : -1, sh = a.sh[p];
  const float* h = a.h + (size_t)p * a.R;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < 16; ++i) d[f][i] = 0.0f;
  uint32_t todo = (uint32_t)__ballot(id >= 0);
  while (todo) {
    const int e = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const uint32_t mine = (uint32_t)__ballot(id == e);
    todo &= ~mine;
    const TX* b[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) b[f] = static_cast<const TX*>(a.ab) + ((size_t)e * a.N + row[f]) * a.R;
    f16v c[2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) c[f][i] = 0.0f;
    if constexpr (std::is_same<TX, float>::value) {
      typedef float f4 __attribute__((ext_vector_type(4)));
      for (int k = 4 * g; k < a.R; k += 8) {  // a rank is a multiple of 8
        f4 hv = *reinterpret_cast<const f4*>(h + k), bv[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) bv[f] = *reinterpret_cast<const f4*>(b[f] + k);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            c[f] = __builtin_amdgcn_mfma_f32_32x32x2f32(ldexpf(hv[j], sh), bv[f][j], c[f], 0, 0, 0);
      }
    } else {
      for (int k0 = 0; k0 < a.R; k0 += 16) {
        const int k = k0 + 8 * g;
        const bool in = k < a.R;
        f8v hv = {};
        b8 hh, hl, bh[2], bl[2];
        if (in) {
          hv = *reinterpret_cast<const f8v*>(h + k);
#pragma unroll
          for (int i = 0; i < 8; ++i) hv[i] = ldexpf(hv[i], sh);
        }
        split_bf16(hv, hh, hl);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          Granule<TX> v = {};
          if (in) load8(b[f] + k, true, v);
          if constexpr (std::is_same<TX, bf16_t>::value) __builtin_memcpy(&bh[f], &v, 16);
          else split_bf16(granule_f32<TX>(v), bh[f], bl[f]);
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          c[f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hl, bh[f], c[f], 0, 0, 0);
          if constexpr (!std::is_same<TX, bf16_t>::value)
            c[f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hh, bl[f], c[f], 0, 0, 0);
          c[f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hh, bh[f], c[f], 0, 0, 0);
        }
      }
    }
    const uint32_t own = mine >> (4 * g);  // bit 8 (i / 4) + i % 4: the position of sum i
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int i = 0; i < 16; ++i) d[f][i] = own >> (8 * (i >> 2) + (i & 3)) & 1 ? c[f][i] : d[f][i];
  }
}

// Parts of a code times what is left of its group scale: for bf16 one fp16 rounding of either is far below the result's own;
// fp16 and fp32 keep the rest of the scale as a second part (fp16 with one: 4.0e-4 off in the 2-norm where the result's
// rounding alone is 2.1e-4).
template <class TX>
constexpr int scaled_parts() {
  return std::is_same<TX, bf16_t>::value ? 1 : 2;
}

// Transposed codes of a step: each lane holds its row's codes of two fragments of 32 columns and needs a column's codes of
// the rows it multiplies. They go through LDS (s_w, [2][64 rows][4 * W bytes]) and are read back transposed, in each group
// of 16 lanes the codes of 16 columns and 16 rows (int8: 8 rows). GF: fragments with group scales of their own, 0 without
// them; WP: parts of a scaled code.
template <int W, int WP, int GF>
__device__ __forceinline__ void unpack_transposed(uint32_t* s_w, const uint32_t (&wn)[2][W], const h8 (&gn)[GF ? GF : 1][WP][2][2],
                                                  h8 (&d)[2][2][2 * WP]) {
  typedef int i2v __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) i2v* lds2;
  const int lane = threadIdx.x & 63, g = lane >> 5, q = lane & 15, ch = lane >> 4 & 1;
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      *reinterpret_cast<u4v*>(s_w + f * 64 * W + lane * W + 4 * i) =
          u4v{wn[f][4 * i], wn[f][4 * i + 1], wn[f][4 * i + 2], wn[f][4 * i + 3]};
  wave_sync();
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (W == 4) {
        const i2v v = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds2)(s_w + f * 256 + (32 * h + 16 * g + q) * 4 + ch * 2));
        d[h][0][f] = codes_h8((uint32_t)v[0]);
        d[h][1][f] = codes_h8((uint32_t)v[1]);
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const i2v v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds2)(s_w + f * 512 + (32 * h + 16 * g + 8 * m + (q >> 1)) * 8 + ch * 4 + (q & 1) * 2));
          d[h][m][f] = codes_h8(__builtin_amdgcn_perm(v[1], v[0], 0x06040200u), __builtin_amdgcn_perm(v[1], v[0], 0x07050301u));
        }
      }
    }
  if constexpr (GF > 0)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const h8 q8 = d[h][m][f];
          d[h][m][f] = q8 * gn[f & (GF - 1)][0][h][m];
          if constexpr (WP == 2) d[h][m][2 + f] = q8 * gn[f & (GF - 1)][1][h][m];
        }
  wave_sync();
}

// KW groups of RW wavefronts: a group's wavefronts take 64 rows each, from wavefront tile wt0 on, the groups share the
// columns.
// Transposed: part `part` of `parts` of the sum goes to `sums` [tokens of the tile][256 columns] where there are several.
template <class TX, int TT, int W, int GSH, int RW, int KW>
__device__ __forceinline__ void tile_run(const LinearArgs& a, int wt0, int t0, char* s_mem, int part = 0, int parts = 1,
                                         float* sums = nullptr) {
  constexpr int NX = std::is_same<TX, float>::value ? 2 : 1;
  constexpr int kStep = NX * TT * 2048;  // halfs of a step: [NX][TT][2 blocks][4 slices][32][8]
  // values that are equal in a wavefront are made so for the compiler: addresses are then a scalar base and a lane's
  // constant offset, without vector arithmetic in the loop
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kLanes = 64 * RW;  // of a group
  const int lane = threadIdx.x & 63, wave = wv % RW, r = lane & 31, g = lane >> 5;
  const int kw = wv / RW, tid = threadIdx.x % kLanes;
  auto s_x = reinterpret_cast<_Float16(*)[kStep]>(s_mem) + kw * 2;
  const int from = kTransposed ? (int)((int64_t)(a.nbp / 2) * part / parts) : 0;
  const int to = kTransposed ? (int)((int64_t)(a.nbp / 2) * (part + 1) / parts) : a.nbp / 2;
  const int steps = (to - from + KW - 1) / KW, p0 = min(from + kw * steps, to), p1 = min(p0 + steps, to);
  const int cols = a.half ? a.half / 32 : (a.N + 63) / 64;  // wavefront tiles over the outputs
  const int wtc = min(wt0 + wave, cols - 1);
  int first[2];  // first weight row (transposed: column) of a fragment
  first[0] = a.half ? wtc * 32 : wtc * 64;
  first[1] = a.half ? a.half + wtc * 32 : wtc * 64 + 32;
  if (kTransposed) first[1] = min(first[1], a.N - 32);
  const uint8_t* src[2];
  const float* ssrc[2];
  const int groups = GSH >= 0 ? (kTransposed ? a.N / 32 : a.nb) >> a.gshift : 0;
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    if (kTransposed) {
      src[f] = a.codes + (size_t)(first[f] / 32) * kTileBlock<W> + (size_t)lane * (4 * W);
      ssrc[f] = nullptr;
    } else {
      src[f] = a.codes + tbw_off<W>(first[f] / 64, 0, a.nb) + (size_t)(first[f] % 64) * (4 * W);
      ssrc[f] = a.scales + (GSH >= 0 ? (size_t)(first[f] / 64) * groups * 64 + first[f] % 64 : (size_t)first[f]);
    }
  }
  // transposed: this wavefront's codes of a step in LDS, [2][64 rows][4 * W bytes], and for each fragment the group scales
  // of a step, [2 blocks][2 halves][2 m][8] halfs in the codes' order
  uint32_t* s_w = reinterpret_cast<uint32_t*>(s_mem + tile_x_lds<TX, TT, RW, KW>()) + wv * (128 * W);
  const size_t step_bytes = kTransposed ? (size_t)(a.N / 32) * kTileBlock<W> : 2 * kTileBlock<W>;
  const _Float16* gsrc[2];
  if constexpr (kTransposed && GSH >= 0)
#pragma unroll
    for (int f = 0; f < 2; ++f) gsrc[f] = a.gs + (size_t)(first[f] / 32 >> a.gshift) * 64 + 16 * g;
  constexpr int kGroupFrags = !kTransposed || GSH < 0 ? 0 : GSH == 0 ? 2 : 1;  // fragments with scales of their own
  constexpr int kWP = kGroupFrags > 0 ? scaled_parts<TX>() : 1;                // parts of a scaled code
  h8 gn[kGroupFrags ? kGroupFrags : 1][kWP][2][2];  // the next step's group scales
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
  h8 wf[2][2][2 * kWP];  // this step's fragments: [block][m][fragment]
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
    if constexpr (kTransposed) {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const u4v* q = reinterpret_cast<const u4v*>(src[f] + (size_t)p * step_bytes);
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const u4v v = q[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) wn[f][4 * i + j] = v[j];
        }
      }
#pragma unroll
      for (int f = 0; f < kGroupFrags; ++f)
#pragma unroll
        for (int v = 0; v < kWP; ++v)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < 2; ++m)
              gn[f][v][h][m] = *reinterpret_cast<const h8*>(gsrc[f] + v * a.gs_low + (size_t)p * groups * 64 + h * 32 + m * 8);
      return;
    }
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
  auto unpack = [&](h8 (&d)[2][2][2 * kWP], float (&ds)[2][kScales]) __attribute__((always_inline)) {
    if constexpr (kTransposed) {
      unpack_transposed<W, kWP, kGroupFrags>(s_w, wn, gn, d);
      return;
    }
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
              if constexpr (GSH < 0 || kTransposed) {
                acc[tt][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, wf[h][m][f], acc[tt][f], 0, 0, 0);
                if constexpr (kWP == 2)
                  if (n == 0) acc[tt][f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, wf[h][m][2 + f], acc[tt][f], 0, 0, 0);
              } else {
                const bool first = m == 0 && n == 0 && (GSH == 0 || h == 0);
                f16v zero;
#pragma unroll
                for (int j = 0; j < 16; ++j) zero[j] = 0.0f;
                c[f] = __builtin_amdgcn_mfma_f32_32x32x16_f16(xf, wf[h][m][f], first ? zero : c[f], 0, 0, 0);
              }
            }
          }
        if constexpr (GSH >= 0 && !kTransposed)
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
      h8 wl[2][2][2 * kWP];
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
          for (int f = 0; f < 2 * kWP; ++f) wf[h][m][f] = wl[h][m][f];
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
  if (GSH < 0 && !kTransposed) rs[0] = ssrc[0][r], rs[1] = ssrc[1][r];
  // results through LDS, 16 tokens at a time, so that they are finished and stored four neighbours a lane
  float* s_out = reinterpret_cast<float*>(s_mem);
  const int rc = column_at<W>(r);
  const int at0 = a.half ? wave * 32 + rc : wave * 64 + rc, at1 = 32 * (a.half ? RW : 1) + at0;
  const int row[2] = {first[0] + rc, first[1] + rc};
  const int quads = (a.half ? 8 : 16) * RW, col0 = wt0 * (a.half ? 32 : 64), out = a.half ? a.half : a.N;
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    f16v d[2];
    if constexpr (kAdapted) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[tt][f][i] *= rs[f];
      if (a.h && kw == 0 && part == 0 && t0 + 32 * tt < a.T) {
        adapter_frags<TX>(a, t0 + 32 * tt, row, lane, d);
#pragma unroll
        for (int f = 0; f < 2; ++f) acc[tt][f] += d[f];
      }
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      __syncthreads();
      if (kw == 0)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int tk = 8 * (i >> 2) + 4 * g + (i & 3);
          s_out[tk * kOutRow + at0] = kAdapted ? acc[tt][0][8 * hh + i] : acc[tt][0][8 * hh + i] * rs[0];
          s_out[tk * kOutRow + at1] = kAdapted ? acc[tt][1][8 * hh + i] : acc[tt][1][8 * hh + i] * rs[1];
        }
      __syncthreads();
      for (int k = threadIdx.x; k < 16 * quads; k += kLanes * KW) {
        const int tk = k / quads, c = k % quads * 4, t = t0 + 32 * tt + 16 * hh + tk;
        if (kTransposed && sums) {
          f4v v = *reinterpret_cast<const f4v*>(s_out + tk * kOutRow + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = ldexpf(v[i], t < a.T ? -a.sh[t] : 0);
          *reinterpret_cast<f4v*>(sums + (size_t)(32 * tt + 16 * hh + tk) * 256 + c) = v;
        } else if (t < a.T && col0 + c < out)
          finish4<TX>(a, token_of(a, t), col0 + c, -a.sh[t], s_out + tk * kOutRow + c,
                      s_out + tk * kOutRow + 32 * RW + c);
      }
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
  return std::is_same<TX, float>::value || GSH == 0 || (GSH > 0 && !(kTransposed && std::is_same<TX, bf16_t>::value)) ? 2 : 4;
}

// Transposed: the sum over the rows in n parts, [n][tiles of the launch][32 * BT tokens][256 columns], added by k_linear_add.
struct TileParts {
  int32_t n;
  float* sums;
};
template <class TX, int TT, int W, int GSH, int RW, int KW>
__global__ __launch_bounds__(64 * RW * KW, RW * KW == 16 ? 4 : 2) void k_linear_tile(LinearArgs a, int row_tiles,
                                                                                     int tok_tiles, int first,
                                                                                     int count, TileParts parts) {
  constexpr int BT = base_frags<TX, GSH>(), kToks = BT / TT, kRows = 4 / RW;  // the cut of a tile
  __shared__ __align__(16) char s_mem[tile_lds<TX, TT, W, RW, KW>()];
  const int n = count * kToks * kRows, d = blockIdx.x % kDies, q = n / kDies, m = n % kDies;
  const int k = d * q + min(d, m) + blockIdx.x / kDies, id = first + k / (kToks * kRows);
  const int group = id / (kTileRowGroup * tok_tiles), in_group = id - group * kTileRowGroup * tok_tiles;
  const int rows_in = min(kTileRowGroup, row_tiles - group * kTileRowGroup);
  const int t0 = in_group / rows_in * 32 * BT + k % kToks * 32 * TT;
  const int wt0 = (group * kTileRowGroup + in_group % rows_in) * 4 + k / kToks % kRows * RW;
  if (t0 >= a.T || wt0 * (a.half ? 32 : 64) >= (a.half ? a.half : a.N)) return;
  if constexpr (kTransposed) {
    const int part = blockIdx.y;
    float* sums = parts.n > 1 ? parts.sums + ((size_t)(part * count + id - first) * 32 * BT + t0 % (32 * BT)) * 256 : nullptr;
    tile_run<TX, TT, W, GSH, RW, KW>(a, wt0, t0, s_mem, part, parts.n, sums);
  } else {
    tile_run<TX, TT, W, GSH, RW, KW>(a, wt0, t0, s_mem);
  }
}

#if !MOE_TRANSPOSED
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
#endif

#if !MOE_TRANSPOSED
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
#endif

// More tokens. What fills the card twice over (two workgroups on each of 256 compute units) runs in whole tiles of four
// wavefronts; of what is left, up to 256 tiles run one a compute unit, with eight wavefronts that share the columns, and
// fewer than that are cut into halves or quarters first. Each step against the one before it, us: 128 x 256 tiles, 256
// of them 103 against 111, 128 44.7 / 62.6, 48 22.0 / 28.1 (2,048 columns; 6,144 42.4 / 71.8), 24 22.0 / 30.6; 64 x 256
// tiles of group scales 384 of them 88 / 87, 192 52.7 / 63.9, 96 39.1 / 50.9, 48 25.6 / 38.5, of fp32 111 / 119, 77 / 75,
// 42 / 74, 30 / 40.
constexpr int kUnits = 256;
#if !MOE_TRANSPOSED
template <class TX, int W, int GSH>
void tile_launch(const LinearArgs& a, float*, hipStream_t st) {
  constexpr int BT = base_frags<TX, GSH>(), KQ = GSH >= 0 ? 2 : 4;
  const int row_tiles = (a.N + 255) / 256, tok_tiles = (a.T + 32 * BT - 1) / (32 * BT);
  const int tiles = row_tiles * tok_tiles;
  for (int at = 0, left; (left = tiles - at) > 0;) {
    if constexpr (BT == 4) {
      if (left >= 2 * kUnits) {
        const int n = left / (2 * kUnits) * (2 * kUnits);
        k_linear_tile<TX, 4, W, GSH, 4, 1><<<n, 256, 0, st>>>(a, row_tiles, tok_tiles, at, n, {});
        at += n;
      } else if (left > kUnits / 2) {
        const int n = std::min(left, kUnits);
        k_linear_tile<TX, 4, W, GSH, 4, 2><<<n, 512, 0, st>>>(a, row_tiles, tok_tiles, at, n, {});
        at += n;
      } else if (left > kUnits / 4) {
        k_linear_tile<TX, 2, W, GSH, 4, 2><<<2 * left, 512, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
        at += left;
      } else if (left > kUnits / 8) {
        k_linear_tile<TX, 1, W, GSH, 4, 4><<<4 * left, 1024, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
        at += left;
      } else {
        k_linear_tile<TX, 1, W, GSH, 2, 8><<<8 * left, 1024, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
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
        k_linear_tile<TX, kWhole ? 2 : 1, W, GSH, 4, 1><<<n, 256, 0, st>>>(a, row_tiles, tok_tiles, at, n, {});
      } else if (left > kUnits) {
        k_linear_tile<TX, 1, W, GSH, 4, 1><<<2 * left, 256, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
      } else if (left > kUnits / 2) {
        k_linear_tile<TX, 2, W, GSH, 4, 2><<<left, 512, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
      } else if (left > kUnits / 4) {
        k_linear_tile<TX, 1, W, GSH, 4, KQ><<<2 * left, 256 * KQ, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
      } else {
        k_linear_tile<TX, 1, W, GSH, 2, 2 * KQ><<<4 * left, 256 * KQ, 0, st>>>(a, row_tiles, tok_tiles, at, left, {});
      }
      at += n;
    }
  }
}
#else
// Adds the parts in ascending order and finishes: a workgroup takes 4 tokens of a tile, a lane 4 columns.
template <class TX, int BT>
__global__ __launch_bounds__(256) void k_linear_add(LinearArgs a, int row_tiles, int tok_tiles, int first, int count,
                                                    TileParts parts) {
  const int id = first + blockIdx.x / (8 * BT), tk = blockIdx.x % (8 * BT) * 4 + (threadIdx.x >> 6);
  const int group = id / (kTileRowGroup * tok_tiles), in_group = id - group * kTileRowGroup * tok_tiles;
  const int rows_in = min(kTileRowGroup, row_tiles - group * kTileRowGroup);
  const int t = in_group / rows_in * 32 * BT + tk, c = (threadIdx.x & 63) * 4;
  const int col = (group * kTileRowGroup + in_group % rows_in) * 256 + c;
  if (t >= a.T || col >= a.N) return;
  const float* p = parts.sums + ((size_t)(id - first) * 32 * BT + tk) * 256 + c;
  const size_t step = (size_t)count * 32 * BT * 256;
  f4v v = *reinterpret_cast<const f4v*>(p);
#pragma unroll 8
  for (int k = 1; k < parts.n; ++k) v += *reinterpret_cast<const f4v*>(p + k * step);
  const float w[4] = {v[0], v[1], v[2], v[3]};
  finish4<TX>(a, token_of(a, t), col, 0, w, w);
}

// As many tiles as fill the card twice over run in workgroups of four wavefronts, up to 256 of the rest with eight that share
// the rows summed over; what is left then, up to 128, is cut into parts of the sum, so that 256 workgroups run again.
// 2,048 tokens, 12288 rows x 6144 columns, bf16: 256 tiles 180 us, the other 128 in two parts 97 and 9 to add, 1.08 PFLOP/s of
// matrix instructions while tiles run (128 as 256 tiles of half the tokens 128 us); bound as the product is, the codes' way
// through LDS hides behind it.
constexpr int kMinSteps = 4;  // of a part
inline int tile_parts(int left, int steps) { return std::max(1, std::min(kUnits / left, steps / kMinSteps)); }
template <class TX, int W, int GSH>
void tile_launch(const LinearArgs& a, float* sums, hipStream_t st) {
  constexpr int BT = base_frags<TX, GSH>();
  const int row_tiles = (a.N + 255) / 256, tok_tiles = (a.T + 32 * BT - 1) / (32 * BT);
  const int tiles = row_tiles * tok_tiles;
  for (int at = 0, left; (left = tiles - at) > 0;) {
    if (left >= 2 * kUnits) {
      const int n = left / (2 * kUnits) * (2 * kUnits);
      k_linear_tile<TX, BT, W, GSH, 4, 1><<<n, 256, 0, st>>>(a, row_tiles, tok_tiles, at, n, {1, nullptr});
      at += n;
    } else if (left > kUnits / 2) {
      const int n = std::min(left, kUnits);
      k_linear_tile<TX, BT, W, GSH, 4, 2><<<n, 512, 0, st>>>(a, row_tiles, tok_tiles, at, n, {1, nullptr});
      at += n;
    } else {
      const TileParts p{tile_parts(left, a.nbp / 2), sums};
      k_linear_tile<TX, BT, W, GSH, 4, 2><<<dim3(left, p.n), 512, 0, st>>>(a, row_tiles, tok_tiles, at, left, p);
      if (p.n > 1) k_linear_add<TX, BT><<<left * 8 * BT, 256, 0, st>>>(a, row_tiles, tok_tiles, at, left, p);
      at += left;
    }
  }
}
// of the parts' sums, for any number of tokens up to T
inline size_t tile_sums_bytes(int N, int steps, int64_t T) {
  const int64_t tiles = (int64_t)((N + 255) / 256) * ((T + 63) / 64);  // the smaller tiles
  return (size_t)std::min<int64_t>(kUnits, tiles * std::max(1, steps / kMinSteps)) * 128 * 256 * 4;
}
#endif

template <class TX>
void tiles_launch(const LinearArgs& a, int bits, float* sums, hipStream_t st) {
  if (bits == 8) tile_launch<TX, 8, -1>(a, sums, st);
  else if (a.gshift < 0) tile_launch<TX, 4, -1>(a, sums, st);
  else if (a.gshift == 0) tile_launch<TX, 4, 0>(a, sums, st);
  else tile_launch<TX, 4, 1>(a, sums, st);
}

#if !MOE_TRANSPOSED
template <class TX>
void few_launch(const LinearArgs& a, int bits, void* ws, hipStream_t st) {
  float* p = static_cast<float*>(ws);
  if (bits == 8) few_tokens<TX, 8, -1>(a, p, st);
  else if (a.gshift < 0) few_tokens<TX, 4, -1>(a, p, st);
  else if (a.gshift == 0) few_tokens<TX, 4, 0>(a, p, st);
  else if (a.gshift == 1) few_tokens<TX, 4, 1>(a, p, st);
  else few_tokens<TX, 4, 2>(a, p, st);
}

template <class TX>
void linear_launch(const LinearArgs& a, int bits, void* ws, hipStream_t st) {
  if (is_slim(a.T, a.N)) {
    few_launch<TX>(a, bits, ws, st);
    return;
  }
  k_linear_x<TX><<<(a.T + 31) / 32 * 4, 8 * kPrepLanes, 0, st>>>(a);
  tiles_launch<TX>(a, bits, nullptr, st);
}

LinearArgs linear_args(const moe_linear_config& c, const uint8_t* codes, const float* scales, const float* bias,
                       const void* x, int64_t ldx, int T, int dtype, const void* res, int64_t ldr, void* y, int64_t ldy,
                       void* ws) {
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
  a.gshift = group_shift(c);
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
  return a;
}
#endif

}  // namespace

}  // namespace moe
