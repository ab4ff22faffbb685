// Rows of bf16 or float32 elements, read and written as float32 in registers.
#pragma once

#include "common.h"
#include "fp8.h"

namespace nvfp4moe {

inline bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

constexpr int64_t kLastLevelCache = 256ll << 20;   // bytes

// 16 bytes; STREAM: non-temporal, for data that the caches would not hold until it is used again
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const void* p) {
  const u32x4* q = static_cast<const u32x4*>(p);
  if constexpr (STREAM) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(q));
  else return __builtin_bit_cast(uint4, *q);
}
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  u32x4* q = static_cast<u32x4*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), q);
  else *q = __builtin_bit_cast(u32x4, v);
}

template <bool STREAM>
__device__ __forceinline__ void store8bytes(void* p, uint2 v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  u32x2* q = static_cast<u32x2*>(p);
  if constexpr (STREAM) __builtin_nontemporal_store((u32x2){v.x, v.y}, q);
  else *q = (u32x2){v.x, v.y};
}

template <bool F32>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return bf16_lo(static_cast<const uint16_t*>(p)[i]);
}

// bf16: rounded to nearest even (a NaN stays one)
template <bool F32>
__device__ __forceinline__ void store_one(void* p, int64_t i, float v) {
  if constexpr (F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)bf16x2_rne(v, 0.0f);
}

// 8 consecutive elements as they lie in memory: one 16-byte word of bf16, two of float32
template <bool F32>
struct Raw8 { uint4 q[F32 ? 2 : 1]; };

template <bool F32, bool STREAM = false>
__device__ __forceinline__ Raw8<F32> load8(const void* p, int64_t i) {
  Raw8<F32> r;
  const char* s = static_cast<const char*>(p) + i * (F32 ? 4 : 2);
#pragma unroll
  for (int j = 0; j < (F32 ? 2 : 1); ++j) r.q[j] = load16<STREAM>(s + 16 * j);
  return r;
}

template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float (&v)[8]) {
  if constexpr (F32) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[2 * j] = bf16_lo(w[j]); v[2 * j + 1] = bf16_hi(w[j]); }
  }
}

// bf16: each value rounded to nearest even
template <bool F32, bool STREAM = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    float* d = static_cast<float*>(p) + i;
#pragma unroll
    for (int j = 0; j < 8; j += 4)
      store16<STREAM>(d + j, make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                                        __float_as_uint(v[j + 3])));
  } else {
    store16<STREAM>(static_cast<uint16_t*>(p) + i, make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]),
                                                              bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])));
  }
}

// the wavefront's sum in every lane, added in a fixed order
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

}  // namespace nvfp4moe
