// linear_types.h — vectors of the matrix instructions, and activations as they lie in memory.
#pragma once

#include <type_traits>

#include "moe_float.h"
#include "moe_ops.h"

namespace moe {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef int i4v __attribute__((ext_vector_type(4)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

// Orders a wavefront's LDS writes before its later reads of other lanes' data.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

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
typedef float f8v __attribute__((ext_vector_type(8)));
template <class TX>
__device__ __forceinline__ f8v granule_f32(const Granule<TX>& d) {
  TX t[8];
  __builtin_memcpy(t, &d, sizeof(d));
  f8v v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32<TX>(t[i]);
  return v;
}

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
// v = hi + lo, 16 bits of it
__device__ __forceinline__ void split_bf16(const f8v& v, b8& hi, b8& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (__bf16)v[i];
    lo[i] = (__bf16)(v[i] - (float)hi[i]);
  }
}

}  // namespace

}  // namespace moe
