// k_clip.hip — the norm over many gradients, and the gradients scaled to a largest norm.
//
// Memory decides: one pass for the norm, one that reads again and writes. A table on the device, written once by the
// caller's program, holds the tensors and which tensor each run of kChunk elements belongs to, so a pass is one launch
// over all of them. Squares are taken and summed in 64 bits: no gradient's square overflows or vanishes. The second
// launch adds the first one's sums itself, in a fixed order.
//
// The second pass goes the other way round, over what the first one left in the card's 256 MB cache, and where all of it
// does not fit (kReread) reads and writes past the caches, which keeps them for the rest of the first pass's and for the
// next one: 100 million fp32 gradients to another array 71 us and 131 (5.7 TB/s read; 1.2 GB in 201 us); in the same
// direction past the caches 65 and 151, with stores through them 103 and 134; 300 million bf16 112 and 221.
#include "linear_types.h"

namespace moe {

namespace {

constexpr int kChunk = 8192;        // elements; 32 of a lane, its loads all in flight
constexpr int kClipBlocks = 2048;   // workgroups at most: eight a compute unit
constexpr int64_t kReread = 4096;   // chunks (128 MB of fp32) that stay in the cache together with their results
constexpr int kTableArgs = 64;      // tensors of a launch that writes the table

struct ClipEntry {
  const void* g;
  void* out;
  int64_t n;
  int64_t first;  // chunk
  int32_t dtype;
  int32_t skip;   // elements between the 16-byte boundary in front of g and g
};
struct ClipHead {
  double sums[kClipBlocks];
};
// table: ClipHead, entries [count], tensor of each chunk [chunks]
struct ClipPlan {
  size_t entries, owner, total;
};
ClipPlan clip_plan(int64_t count, int64_t chunks) {
  ClipPlan p;
  p.entries = sizeof(ClipHead);
  p.owner = p.entries + (size_t)count * sizeof(ClipEntry);
  p.total = (p.owner + (size_t)chunks * 4 + 255) & ~(size_t)255;
  return p;
}
size_t size_of(int32_t dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }
int32_t skip_of(const moe_grad& g) { return (int32_t)(reinterpret_cast<uintptr_t>(g.g) % 16 / size_of(g.dtype)); }
int64_t chunks_of(const moe_grad& g) { return g.n == 0 ? 0 : (g.n + skip_of(g) + kChunk - 1) / kChunk; }

struct TableArgs {
  ClipEntry e[kTableArgs];
  int32_t first;
  ClipEntry* entries;
  int32_t* owner;
};
// a workgroup for each tensor
__global__ __launch_bounds__(256) void k_clip_table(TableArgs a) {
  const ClipEntry e = a.e[blockIdx.x];
  if (threadIdx.x == 0) a.entries[a.first + blockIdx.x] = e;
  const int64_t chunks = e.n == 0 ? 0 : (e.n + e.skip + kChunk - 1) / kChunk;
  for (int64_t k = threadIdx.x; k < chunks; k += 256) a.owner[e.first + k] = a.first + blockIdx.x;
}

// Addresses that come from the table are of global memory (the compiler cannot see it and would take flat accesses).
template <class T>
using Global = __attribute__((address_space(1))) T;

// f(index of the first element, vector) for the vectors of a chunk, lane's k-th is 256 k + tid: elements are numbered from
// the 16-byte boundary in front of the tensor, and those in front of it and behind it are 0 and not read. LAST: nobody reads
// them again soon, so that they pass by the caches.
template <class T, bool LAST, class F>
__device__ __forceinline__ void each_vector(const ClipEntry& e, int64_t chunk, F&& f) {
  constexpr int V = 16 / sizeof(T), kPer = kChunk / (256 * V);
  const int64_t first = chunk * kChunk, end = e.n + e.skip;
  const Global<const T>* g = (const Global<const T>*)(static_cast<const T*>(e.g) - e.skip) + first;
  u4v d[kPer];
  if (first >= e.skip && first + kChunk <= end) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const Global<const u4v>* at = (const Global<const u4v>*)g + 256 * k + threadIdx.x;
      d[k] = LAST ? __builtin_nontemporal_load(at) : *at;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      T t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int at = (256 * k + threadIdx.x) * V + i;
        t[i] = from_f32<T>(0.0f);
        if (first + at >= e.skip && first + at < end) __builtin_memcpy(&t[i], g + at, sizeof(T));
      }
      d[k] = __builtin_bit_cast(u4v, t);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) f(first + (256 * k + threadIdx.x) * V, d[k]);
}

template <class T>
__device__ __forceinline__ double squares(const ClipEntry& e, int64_t chunk) {
  double s = 0.0;
  each_vector<T, false>(e, chunk, [&](int64_t, const u4v& d) __attribute__((always_inline)) {
    T t[16 / sizeof(T)];
    __builtin_memcpy(t, &d, 16);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i) {
      const double v = (double)to_f32<T>(t[i]);
      s = fma(v, v, s);
    }
  });
  return s;
}

__device__ __forceinline__ double block_sum(double v, double* s_wave) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = v;
  __syncthreads();
  return s_wave[0] + s_wave[1] + s_wave[2] + s_wave[3];
}

__global__ __launch_bounds__(256) void k_clip_norm(const ClipEntry* __restrict__ entries, const int32_t* __restrict__ owner,
                                                   int64_t chunks, double* __restrict__ sums) {
  __shared__ double s_wave[4];
  double s = 0.0;
  ClipEntry next{};
  if (chunks > 0) next = entries[owner[min((int64_t)blockIdx.x, chunks - 1)]];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const ClipEntry e = next;
    const int64_t after = min(c + gridDim.x, chunks - 1);
    const int32_t who = owner[after];
    if (e.dtype == MOE_DTYPE_F32) s += squares<float>(e, c - e.first);
    else if (e.dtype == MOE_DTYPE_BF16) s += squares<bf16_t>(e, c - e.first);
    else s += squares<_Float16>(e, c - e.first);
    next = entries[who];
  }
  s = block_sum(s, s_wave);
  if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// out = g factor 2^exp, in this order. FAR: exp is not 0, see k_clip_scale.
template <class T, bool LAST, bool FAR>
__device__ __forceinline__ void scale_chunk(const ClipEntry& e, int64_t chunk, float factor, int exp) {
  constexpr int V = 16 / sizeof(T);
  Global<T>* out = (Global<T>*)(static_cast<T*>(e.out) - e.skip);
  const bool whole = (uintptr_t)out % 16 == 0;
  const int64_t end = e.n + e.skip;
  each_vector<T, LAST>(e, chunk, [&](int64_t at, const u4v& d) __attribute__((always_inline)) {
    T t[V];
    __builtin_memcpy(t, &d, 16);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = to_f32<T>(t[i]) * factor;
      t[i] = from_f32<T>(FAR ? __builtin_amdgcn_ldexpf(v, exp) : v);
    }
    if (whole && at >= e.skip && at + V <= end) {
      Global<u4v>* to = (Global<u4v>*)(out + at);
      if (LAST) __builtin_nontemporal_store(__builtin_bit_cast(u4v, t), to);
      else *to = __builtin_bit_cast(u4v, t);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at + i >= e.skip && at + i < end) __builtin_memcpy(out + at + i, &t[i], sizeof(T));
    }
  });
}

template <bool LAST>
__global__ __launch_bounds__(256) void k_clip_scale(const ClipEntry* __restrict__ entries, const int32_t* __restrict__ owner,
                                                    int64_t chunks, const double* __restrict__ sums, int count,
                                                    float max_norm, float* __restrict__ norm) {
  __shared__ double s_wave[4];
  ClipEntry next{};
  if (chunks > 0) next = entries[owner[max(chunks - 1 - (int64_t)blockIdx.x, (int64_t)0)]];
  double v[kClipBlocks / 256];
#pragma unroll
  for (int k = 0; k < kClipBlocks / 256; ++k) {
    const int i = 256 * k + threadIdx.x;
    v[k] = i < count ? sums[i] : 0.0;
  }
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kClipBlocks / 256; ++k) s += v[k];
  const double n = sqrt(block_sum(s, s_wave));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
  // an infinite or NaN norm leaves the gradients as they are
  const double ratio = n > (double)max_norm && (float)n < INFINITY ? (double)max_norm / n : 1.0;
  // A factor below fp32's normal range would lose bits, or be 0: its power of two is applied behind the product. (For every
  // factor that takes 335 us where 300 million bf16 gradients take 329.)
  const bool far = ratio < 0x1p-126;
  const int exp = far ? __builtin_amdgcn_frexp_exp(ratio) : 0;
  const float factor = (float)(far ? __builtin_amdgcn_frexp_mant(ratio) : ratio);
  auto scale = [&](const ClipEntry& e, int64_t chunk, auto type) __attribute__((always_inline)) {
    if (far) scale_chunk<decltype(type), LAST, true>(e, chunk, factor, exp);
    else scale_chunk<decltype(type), LAST, false>(e, chunk, factor, 0);
  };
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const ClipEntry e = next;
    const int32_t who = owner[max(chunks - 1 - c - gridDim.x, (int64_t)0)];
    if (factor != 1.0f || e.out != e.g) {
      const int64_t at = chunks - 1 - c - e.first;
      if (e.dtype == MOE_DTYPE_F32) scale(e, at, float());
      else if (e.dtype == MOE_DTYPE_BF16) scale(e, at, bf16_t());
      else scale(e, at, _Float16());
    }
    next = entries[who];
  }
}

}  // namespace

int64_t clip_chunks(const moe_grad* g, int count) {
  int64_t n = 0;
  for (int i = 0; i < count; ++i) n += chunks_of(g[i]);
  return n;
}
size_t clip_table_bytes(const moe_grad* g, int count) { return clip_plan(count, clip_chunks(g, count)).total; }

hipError_t launch_clip_table(const moe_grad* g, int count, void* table, hipStream_t st) {
  const ClipPlan p = clip_plan(count, clip_chunks(g, count));
  char* w = static_cast<char*>(table);
  int64_t chunk = 0;
  for (int at = 0; at < count; at += kTableArgs) {
    TableArgs a;
    a.first = at;
    const int n = count - at < kTableArgs ? count - at : kTableArgs;
    a.entries = reinterpret_cast<ClipEntry*>(w + p.entries);
    a.owner = reinterpret_cast<int32_t*>(w + p.owner);
    for (int i = 0; i < n; ++i) {
      a.e[i] = ClipEntry{g[at + i].g, g[at + i].out, g[at + i].n, chunk, g[at + i].dtype, skip_of(g[at + i])};
      chunk += chunks_of(g[at + i]);
    }
    k_clip_table<<<n, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_clip(const moe_grads& t, float max_norm, float* norm, hipStream_t st) {
  const ClipPlan p = clip_plan(t.count, t.chunks);
  char* w = static_cast<char*>(t.table);
  double* sums = reinterpret_cast<double*>(w);
  const ClipEntry* entries = reinterpret_cast<const ClipEntry*>(w + p.entries);
  const int32_t* owner = reinterpret_cast<const int32_t*>(w + p.owner);
  const int blocks = (int)(t.chunks < 1 ? 1 : t.chunks < kClipBlocks ? t.chunks : kClipBlocks);
  k_clip_norm<<<blocks, 256, 0, st>>>(entries, owner, t.chunks, sums);
  if (t.chunks > kReread) {
    k_clip_scale<true><<<blocks, 256, 0, st>>>(entries, owner, t.chunks, sums, blocks, max_norm, norm);
  } else {
    k_clip_scale<false><<<blocks, 256, 0, st>>>(entries, owner, t.chunks, sums, blocks, max_norm, norm);
  }
  return hipGetLastError();
}

}  // namespace moe
