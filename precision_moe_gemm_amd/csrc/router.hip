// The router's choice (top-k experts of each token and their weights) and its gradient, for gfx950.
// One wavefront per token; lane l holds the experts [l NE, (l + 1) NE) of the row in registers.
#include "common.h"
#include "fp8.h"
#include "rows.h"

namespace nvfp4moe {
namespace router {

constexpr int kWaves = 4;   // wavefronts (tokens) per 256-thread workgroup

// A float's place in the router's order as an unsigned word: larger logits have larger words, both zeros
// the same one, and a NaN the largest.  0 is no logit's word.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
  if (v != v) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t w) {
  if (w == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((w & 0x80000000u) ? (w & 0x7FFFFFFFu) : ~w);
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, kWave));
  return v;
}

// exp(v - m) of the softmax with maximum m: 0 everywhere in a row of -inf alone, NaN where the maximum
// is +inf or NaN.
__device__ __forceinline__ float exp_from(float v, float m) {
  return m == -INFINITY ? 0.0f : expf(v - m);
}

// The k largest logits of each row, equal ones by their index: k rounds of a wavefront maximum over the
// lanes' own maxima.  The lanes hold consecutive experts, so that the first lane with the maximum, and the
// first of its equal ones, is the lowest index.  Lane s keeps the choice of round s.
template <int NE, bool F32>
__global__ __launch_bounds__(kWaves * 64) void topk_kernel(const void* __restrict__ logits, int64_t T, int E, int k,
                                                           int renorm, int32_t* __restrict__ ids, float* __restrict__ w) {
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = lane_id();
  float v[NE];
  uint32_t key[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane * NE + j;
    v[j] = e < E ? load_one<F32>(logits, t * E + e) : 0.0f;
    key[j] = e < E ? order_of(v[j]) : 0u;
  }
  int id = 0;
  uint32_t picked = 0;
  for (int s = 0; s < k; ++s) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int j = 1; j < NE; ++j)
      if (key[j] > best) { best = key[j]; at = j; }
    const uint32_t most = wave_max_u32(best);
    const int from = __ffsll((unsigned long long)__ballot(best == most)) - 1;
    const int e = __shfl(lane * NE + at, from, kWave);
    if (lane == s) { id = e; picked = most; }
    if (lane == from) {
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (j == at) key[j] = 0u;
    }
  }
  const float m = __shfl(of_order(picked), 0, kWave);
  const float mine = lane < k ? exp_from(of_order(picked), m) : 0.0f;
  float sum = mine;
  if (!renorm) {
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (lane * NE + j < E) sum += exp_from(v[j], m);
  }
  sum = wave_sum(sum);
  if (lane < k) {
    ids[t * k + lane] = id;
    w[t * k + lane] = m == -INFINITY ? 0.0f : mine / sum;
  }
}

// The logits' gradient from the weights' g: with mean = sum_s w_s g_s over the token's entries,
//   renorm: dl_e = sum over the entries s of e of w_s (g_s - mean), 0 for an expert that was not chosen;
//   else    dl_e = p_e (sum over the entries s of e of g_s - mean), p = softmax of the row.
template <int NE, bool F32>
__global__ __launch_bounds__(kWaves * 64) void topk_backward_kernel(
    const void* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, int64_t T, int E, int k, int renorm, void* __restrict__ dlogits) {
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = lane_id();
  int id = -1;
  float ws = 0.0f, g = 0.0f;
  if (lane < k) {
    id = ids[t * k + lane];
    if (id >= 0 && id < E) { ws = w[t * k + lane]; g = dw[t * k + lane]; }
    else id = -1;
  }
  const float mean = wave_sum(ws * g);
  const float mine = renorm ? ws * (g - mean) : g;
  float sum[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) sum[j] = 0.0f;
  for (int s = 0; s < k; ++s) {
    const int e = __shfl(id, s, kWave);
    const float x = __shfl(mine, s, kWave);
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (e == lane * NE + j) sum[j] += x;
  }
  if (!renorm) {
    float v[NE], m = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const int e = lane * NE + j;
      v[j] = e < E ? load_one<F32>(logits, t * E + e) : -INFINITY;
      nan |= v[j] != v[j];
      m = fmaxf(m, v[j]);
    }
    m = wave_max(m);
    if (__ballot(nan)) m = NAN;
    float total = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      v[j] = exp_from(v[j], m);
      total += v[j];
    }
    total = wave_sum(total);
#pragma unroll
    for (int j = 0; j < NE; ++j) sum[j] = m == -INFINITY ? 0.0f : v[j] / total * (sum[j] - mean);
  }
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int e = lane * NE + j;
    if (e < E) store_one<F32>(dlogits, t * E + e, sum[j]);
  }
}

inline int check(int64_t T, int32_t E, int32_t k, int32_t dtype, int32_t renorm) {
  if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_ARG;
  if (renorm != 0 && renorm != 1) return NVFP4_ERR_ARG;
  if (T < 0 || E < 1 || E > NVFP4MOE_MAX_EXPERTS || k < 1 || k > E || k > NVFP4MOE_MAX_TOPK) return NVFP4_ERR_SHAPE;
  if (T * (int64_t)k > INT32_MAX / 2) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

}  // namespace router
}  // namespace nvfp4moe

using namespace nvfp4moe;

#define ROUTER_DISPATCH(KERNEL, ...)                                                        \
  do {                                                                                      \
    const unsigned grid = (unsigned)((T + router::kWaves - 1) / router::kWaves);            \
    const bool f32 = dtype == NVFP4_IN_F32;                                                 \
    hipStream_t s = static_cast<hipStream_t>(stream);                                       \
    if (E <= 64) f32 ? KERNEL<1, true><<<grid, 256, 0, s>>>(__VA_ARGS__) : KERNEL<1, false><<<grid, 256, 0, s>>>(__VA_ARGS__);        \
    else if (E <= 128) f32 ? KERNEL<2, true><<<grid, 256, 0, s>>>(__VA_ARGS__) : KERNEL<2, false><<<grid, 256, 0, s>>>(__VA_ARGS__);  \
    else if (E <= 256) f32 ? KERNEL<4, true><<<grid, 256, 0, s>>>(__VA_ARGS__) : KERNEL<4, false><<<grid, 256, 0, s>>>(__VA_ARGS__);  \
    else if (E <= 512) f32 ? KERNEL<8, true><<<grid, 256, 0, s>>>(__VA_ARGS__) : KERNEL<8, false><<<grid, 256, 0, s>>>(__VA_ARGS__);  \
    else f32 ? KERNEL<16, true><<<grid, 256, 0, s>>>(__VA_ARGS__) : KERNEL<16, false><<<grid, 256, 0, s>>>(__VA_ARGS__);              \
  } while (0)

extern "C" {

NVFP4MOE_API int moe_router_topk(const void* logits, int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t renorm,
                                 int32_t* topk_ids, float* topk_w, void* stream) {
  if (const int bad = router::check(T, E, k, dtype, renorm)) return bad;
  if (T == 0) return NVFP4_OK;
  if (!logits || !topk_ids || !topk_w) return NVFP4_ERR_NULL;
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(topk_w)) return NVFP4_ERR_ALIGN;
  ROUTER_DISPATCH(router::topk_kernel, logits, T, (int)E, (int)k, (int)renorm, topk_ids, topk_w);
  return launch_status();
}

NVFP4MOE_API int moe_router_topk_backward(const void* logits, int32_t dtype, const int32_t* topk_ids,
                                          const float* topk_w, const float* dtopk_w, int64_t T, int32_t E, int32_t k,
                                          int32_t renorm, void* dlogits, void* stream) {
  if (const int bad = router::check(T, E, k, dtype, renorm)) return bad;
  if (T == 0) return NVFP4_OK;
  if (!topk_ids || !topk_w || !dtopk_w || !dlogits || (!renorm && !logits)) return NVFP4_ERR_NULL;
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(topk_w) || !aligned16(dtopk_w) || !aligned16(dlogits))
    return NVFP4_ERR_ALIGN;
  if (dlogits == logits) return NVFP4_ERR_ARG;
  ROUTER_DISPATCH(router::topk_backward_kernel, logits, topk_ids, topk_w, dtopk_w, T, (int)E, (int)k, (int)renorm, dlogits);
  return launch_status();
}

}  // extern "C"
