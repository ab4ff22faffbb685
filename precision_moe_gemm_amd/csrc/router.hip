// The router's choice (top-k experts of each token and their weights) and its gradient, for gfx950.
//
// A group of G lanes takes a token: G = 16 (four tokens a wavefront) up to 256 experts, the whole wavefront
// above.  Each lane holds NE consecutive logits, read as vectors wherever the row starts.  A round of the
// choice costs a group's reduction whatever the group's size, so that more tokens share it in the narrow
// groups: 16381 x 250 bf16 logits, k = 6, take 6.6 us for 13.7 with a wavefront a token (8.2 MB read: 1.6 us
// at a copy's rate), the gradient 8.3 for 11.8 (16.4 MB).  Of these a launch of one token takes 3.5 and 2.4,
// the chain of its loads, rounds and stores.  Up to two wavefronts a SIMD run little more than one such chain;
// beyond, the issue of their instructions shows (some 800 each, 4 cycles an instruction: 1.35 us a wavefront on a
// SIMD): launches in a row in a graph, over all experts, take 4.9 us at one token, 5.1, 5.4, 5.6 and 5.9 at 1024,
// 2048, 4096 and 8192, 7.8 at 16381, the gradient 5.2, 5.6, 5.7, 5.9, 7.1 and 10.0, with renorm 4.8, 4.7, 5.4, 5.4,
// 5.6 and 6.2.  Windows of 32 in narrow groups up to 512 experts: 8192 x 512 bf16 5.7 us for 7.3, but float32 with
// its gradient 13.7 + 13.7 for 13.5 + 9.9.
#include "common.h"
#include "fp8.h"
#include "rows.h"

namespace nvfp4moe {
namespace router {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ groups of 16 or 64 lanes
template <int ROR>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {   // within the 16 lanes of a row
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + ROR, 0xF, 0xF, true);
}
template <int ROR>
__device__ __forceinline__ float rotated(float v) { return __uint_as_float(rotated<ROR>(__float_as_uint(v))); }
template <int ROR>
__device__ __forceinline__ double rotated(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint64_t r = ((uint64_t)rotated<ROR>((uint32_t)(b >> 32)) << 32) | rotated<ROR>((uint32_t)b);
  return __longlong_as_double((long long)r);
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }

// The group's maximum, and its sum (the same bits in every lane: each step adds the same two numbers on
// both sides), in every lane.
template <int G, class V>
__device__ __forceinline__ V group_max(V v) {
  v = larger(v, rotated<8>(v));
  v = larger(v, rotated<4>(v));
  v = larger(v, rotated<2>(v));
  v = larger(v, rotated<1>(v));
  if constexpr (G == 64) {
    v = larger(v, (V)__shfl_xor(v, 16, kWave));
    v = larger(v, (V)__shfl_xor(v, 32, kWave));
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += rotated<8>(v);
  v += rotated<4>(v);
  v += rotated<2>(v);
  v += rotated<1>(v);
  if constexpr (G == 64) {
    v += __shfl_xor(v, 16, kWave);
    v += __shfl_xor(v, 32, kWave);
  }
  return v;
}

// ------------------------------------------------------------------ a lane's logits
// Lane g of a group holds the experts [g NE, (g + 1) NE) of E >= NE.  The lanes at the row's end read
// the row's last NE logits, so that no lane reads beside the row and every one reads whole vectors; of
// these, an expert below g NE is another lane's.
template <int NE>
__device__ __forceinline__ int window(int g, int E) { return min(g * NE, E - NE); }

template <int NE, bool F32>
__device__ __forceinline__ void load_logits(const void* logits, int64_t at, float (&v)[NE]) {
  if constexpr (F32) {
    __builtin_memcpy(v, static_cast<const float*>(logits) + at, NE * 4);
  } else {
    uint16_t b[NE];
    __builtin_memcpy(b, static_cast<const uint16_t*>(logits) + at, NE * 2);
#pragma unroll
    for (int j = 0; j < NE; ++j) v[j] = bf16_lo(b[j]);
  }
}

template <int NE, bool F32>
__device__ __forceinline__ void store_logits(void* dlogits, int64_t at, const float (&v)[NE]) {
  if constexpr (F32) {
    __builtin_memcpy(static_cast<float*>(dlogits) + at, v, NE * 4);
  } else if constexpr (NE == 1) {
    store_one<false>(dlogits, at, v[0]);
  } else {
    uint32_t b[NE / 2];
#pragma unroll
    for (int j = 0; j < NE / 2; ++j) b[j] = bf16x2_rne(v[2 * j], v[2 * j + 1]);
    __builtin_memcpy(static_cast<uint16_t*>(dlogits) + at, b, NE * 2);
  }
}

// A float's place in the router's order as an unsigned word: larger logits have larger words, both zeros
// the same one, and a NaN the largest.  0 is no logit's word.  A bf16's is in the upper half.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
  if (v != v) return 0xFFFFFFFFu;
  return u ^ (uint32_t)(((int32_t)u >> 31) | (int32_t)0x80000000);
}
__device__ __forceinline__ float of_order(uint32_t w, uint32_t nan) {
  if (w == nan) return NAN;
  return __uint_as_float(((w & 0x80000000u) ? w ^ 0x80000000u : ~w) & nan);
}

// The candidates of a lane: each logit's word above its expert's number counted down, so that the largest
// is the largest logit, of equal ones the lowest expert's, and no two are alike.  next() is the group's
// largest one below those already given.
//
// bf16: 16 + 16 bits.  With d_j = key_j - last modulo 2^32, the keys below `last` have the largest d, in
// their own order: one subtraction and half a three-operand maximum a key, nothing to be taken out.
template <int NE, int G, bool F32>
struct Keys {
  uint32_t key[NE], last = 0;
  __device__ __forceinline__ void set(int j, float v, int e, bool mine) {
    key[j] = mine ? (order_of(v) & 0xFFFF0000u) | (0xFFFFu - (uint32_t)e) : 0u;
  }
  __device__ __forceinline__ void next(float& v, int& e) {
    uint32_t d = key[0] - last;
#pragma unroll
    for (int j = 1; j < NE; ++j) d = max(d, key[j] - last);
    last += group_max<G>(d);
    v = of_order(last & 0xFFFF0000u, 0xFFFF0000u);
    e = (int)(0xFFFFu - (last & 0xFFFFu));
  }
};

// float32: 32 + 10 bits in the mantissa of a float64 between 1 and 2, whose maxima are single instructions;
// the one that was given is taken out (without its upper word it is below them all).
template <int NE, int G>
struct Keys<NE, G, true> {
  double key[NE];
  __device__ __forceinline__ void set(int j, float v, int e, bool mine) {
    const uint64_t b = (1023ull << 52) | ((uint64_t)order_of(v) << 10) | (uint64_t)(1023 - e);
    key[j] = mine ? __longlong_as_double((long long)b) : 0.0;
  }
  __device__ __forceinline__ void next(float& v, int& e) {
    double d = key[0];
#pragma unroll
    for (int j = 1; j < NE; ++j) d = larger(d, key[j]);
    d = group_max<G>(d);
    const uint64_t b = (uint64_t)__double_as_longlong(d);
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const uint64_t c = (uint64_t)__double_as_longlong(key[j]);
      key[j] = __longlong_as_double((long long)(((uint64_t)(c == b ? 0u : (uint32_t)(c >> 32)) << 32) | (uint32_t)c));
    }
    v = of_order((uint32_t)(b >> 10), 0xFFFFFFFFu);
    e = 1023 - (int)(b & 1023u);
  }
};

// exp(v - m) of the softmax with maximum m.  A row of -inf alone has the sum 0, and weights of 0; where the
// row holds a NaN or +inf, the sum is NaN.
__device__ __forceinline__ float exp_from(float v, float m) { return v == -INFINITY ? 0.0f : expf(v - m); }
__device__ __forceinline__ float part_of(float e, float sum) { return sum == 0.0f ? 0.0f : e / sum; }

// The k largest logits of each row in k rounds; lane s modulo G keeps the choice of round s.
template <int NE, int G, bool F32>
__global__ __launch_bounds__(kThreads) void topk_kernel(const void* __restrict__ logits, int64_t T, int E, int k,
                                                        int renorm, int32_t* __restrict__ ids, float* __restrict__ w) {
  constexpr int kSlots = (NVFP4MOE_MAX_TOPK + G - 1) / G;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const int64_t t = min(row, T - 1);              // groups past the last token read it again
  const int g = threadIdx.x % G, from = window<NE>(g, E);
  float v[NE];
  load_logits<NE, F32>(logits, t * E + from, v);
  Keys<NE, G, F32> keys;
#pragma unroll
  for (int j = 0; j < NE; ++j) keys.set(j, v[j], from + j, from + j >= g * NE);
  float m = 0.0f, pv[kSlots];
  int pe[kSlots];
#pragma unroll
  for (int u = 0; u < kSlots; ++u) { pv[u] = -INFINITY; pe[u] = 0; }
  for (int s = 0; s < k; ++s) {
    float x;
    int e;
    keys.next(x, e);
    if (s == 0) m = x;
#pragma unroll
    for (int u = 0; u < kSlots; ++u)
      if (s == u * G + g) { pv[u] = x; pe[u] = e; }
  }
  float sum = 0.0f;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    pv[u] = exp_from(pv[u], m);
    sum += pv[u];
  }
  if (!renorm) {
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j) sum += from + j >= g * NE ? exp_from(v[j], m) : 0.0f;
  }
  sum = group_sum<G>(sum);
  if (row >= T) return;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    const int s = u * G + g;
    if (s < k) {
      ids[t * k + s] = pe[u];
      w[t * k + s] = part_of(pv[u], sum);
    }
  }
}

// The logits' gradient from the weights' g: with mean = sum_s w_s g_s over the token's entries,
//   renorm: dl_e = sum over the entries s of e of w_s (g_s - mean), 0 for an expert that was not chosen;
//   else    dl_e = p_e (sum over the entries s of e of g_s - mean), p = softmax of the row.
// An expert's sum goes to the lane that holds the expert through the row's line in LDS (a word of padding a
// lane keeps the lanes' words in different banks).  Each entry first leaves its number there: one that reads
// another's back shares its expert, and then the sums over equal experts are formed, in slot order, by the
// first entry of each; a router's choices are all different, and their sums the entries' own.
template <int NE, int G, bool F32>
__global__ __launch_bounds__(kThreads) void topk_backward_kernel(
    const void* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ w,
    const float* __restrict__ dw, int64_t T, int E, int k, int renorm, void* __restrict__ dlogits) {
  constexpr int kSlots = (NVFP4MOE_MAX_TOPK + G - 1) / G;
  constexpr int kLine = NE * G + G;
  __shared__ float lines[kThreads / G][kLine];
  const int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const int64_t t = min(row, T - 1);
  const int g = threadIdx.x % G, from = window<NE>(g, E);
  float* line = lines[threadIdx.x / G];
  const auto at = [](int e) { return e + e / NE; };
  float v[NE];
  if (!renorm) load_logits<NE, F32>(logits, t * E + from, v);
  int id[kSlots];
  float x[kSlots], ws[kSlots];
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    const int64_t i = t * k + min(u * G + g, k - 1);
    id[u] = ids[i];
    ws[u] = w[i];
    x[u] = dw[i];
  }
#pragma unroll
  for (int j = 0; j < kLine; j += G) line[j + g] = 0.0f;
  __syncthreads();
  float mean = 0.0f;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    if (u * G + g >= k || id[u] < 0 || id[u] >= E) { id[u] = -1; ws[u] = x[u] = 0.0f; }
    mean += ws[u] * x[u];
    if (id[u] >= 0) line[at(id[u])] = __int_as_float(u * G + g);
  }
  mean = group_sum<G>(mean);
  __syncthreads();
  float total[kSlots];
  bool first[kSlots], shared = false;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    if (renorm) x[u] = ws[u] * (x[u] - mean);
    total[u] = x[u];
    first[u] = id[u] >= 0;
    shared |= first[u] && __float_as_int(line[at(id[u])]) != u * G + g;
  }
  if (__ballot(shared)) {
#pragma unroll
    for (int u = 0; u < kSlots; ++u) total[u] = 0.0f;
    for (int q = 0; q < k; ++q) {
      const bool hi = q >= G;
      const int e = __shfl(hi ? id[kSlots - 1] : id[0], q % G, G);
      const float y = __shfl(hi ? x[kSlots - 1] : x[0], q % G, G);
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (e != id[u]) continue;
        total[u] += y;
        if (q < u * G + g) first[u] = false;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kSlots; ++u)
    if (first[u]) line[at(id[u])] = total[u];
  __syncthreads();
  float d[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) d[j] = line[at(from + j)];
  if (!renorm) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < NE; ++j) m = fmaxf(m, v[j]);
    m = group_max<G>(m);                          // of the numbers; a NaN reaches the sum
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      v[j] = exp_from(v[j], m);
      sum += from + j >= g * NE ? v[j] : 0.0f;
    }
    sum = group_sum<G>(sum);
#pragma unroll
    for (int j = 0; j < NE; ++j) d[j] = part_of(v[j], sum) * (d[j] - mean);
  }
  if (row < T && g * NE < E) store_logits<NE, F32>(dlogits, t * E + from, d);   // windows that overlap hold the same bits
}

inline int check(int64_t T, int32_t E, int32_t k, int32_t dtype, int32_t renorm) {
  if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_ARG;
  if (renorm != 0 && renorm != 1) return NVFP4_ERR_ARG;
  if (T < 0 || E < 1 || E > NVFP4MOE_MAX_EXPERTS || k < 1 || k > E || k > NVFP4MOE_MAX_TOPK) return NVFP4_ERR_SHAPE;
  return T > MOE_MAX_ROWS || T * (int64_t)k > MOE_MAX_ROWS ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

}  // namespace router
}  // namespace nvfp4moe

using namespace nvfp4moe;

// The narrowest group, and in it the shortest windows, that hold E experts (every window is at most E).
#define ROUTER_LAUNCH(KERNEL, NE, G, ...)                                                                   \
  do {                                                                                                      \
    const unsigned grid = (unsigned)((T + router::kThreads / (G) - 1) / (router::kThreads / (G)));          \
    if (dtype == NVFP4_IN_F32) KERNEL<NE, G, true><<<grid, router::kThreads, 0, s>>>(__VA_ARGS__);          \
    else KERNEL<NE, G, false><<<grid, router::kThreads, 0, s>>>(__VA_ARGS__);                               \
  } while (0)
#define ROUTER_DISPATCH(KERNEL, ...)                                     \
  do {                                                                   \
    hipStream_t s = static_cast<hipStream_t>(stream);                    \
    if (E <= 16) ROUTER_LAUNCH(KERNEL, 1, 16, __VA_ARGS__);              \
    else if (E <= 64) ROUTER_LAUNCH(KERNEL, 4, 16, __VA_ARGS__);         \
    else if (E <= 128) ROUTER_LAUNCH(KERNEL, 8, 16, __VA_ARGS__);        \
    else if (E <= 256) ROUTER_LAUNCH(KERNEL, 16, 16, __VA_ARGS__);       \
    else if (E <= 512) ROUTER_LAUNCH(KERNEL, 8, 64, __VA_ARGS__);        \
    else ROUTER_LAUNCH(KERNEL, 16, 64, __VA_ARGS__);                     \
  } while (0)

extern "C" {

NVFP4MOE_API int moe_router_topk(const void* logits, int32_t dtype, int64_t T, int32_t E, int32_t k, int32_t renorm,
                                 int32_t* topk_ids, float* topk_w, void* stream) {
  if (const int bad = router::check(T, E, k, dtype, renorm)) return bad;
  if (T == 0) return NVFP4_OK;
  if (!logits || !topk_ids || !topk_w) return NVFP4_ERR_NULL;
  if (!aligned_to(logits, dtype == NVFP4_IN_F32 ? 4 : 2) || !aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4))
    return NVFP4_ERR_ALIGN;
  ROUTER_DISPATCH(router::topk_kernel, logits, T, (int)E, (int)k, (int)renorm, topk_ids, topk_w);
  return launch_status();
}

NVFP4MOE_API int moe_router_topk_backward(const void* logits, int32_t dtype, const int32_t* topk_ids,
                                          const float* topk_w, const float* dtopk_w, int64_t T, int32_t E, int32_t k,
                                          int32_t renorm, void* dlogits, void* stream) {
  if (const int bad = router::check(T, E, k, dtype, renorm)) return bad;
  if (T == 0) return NVFP4_OK;
  if (!topk_ids || !topk_w || !dtopk_w || !dlogits || (!renorm && !logits)) return NVFP4_ERR_NULL;
  const int size = dtype == NVFP4_IN_F32 ? 4 : 2;
  if (!aligned_to(logits, size) || !aligned_to(dlogits, size) || !aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4) ||
      !aligned_to(dtopk_w, 4))
    return NVFP4_ERR_ALIGN;
  if (dlogits == logits) return NVFP4_ERR_ARG;
  ROUTER_DISPATCH(router::topk_backward_kernel, logits, topk_ids, topk_w, dtopk_w, T, (int)E, (int)k, (int)renorm, dlogits);
  return launch_status();
}

}  // extern "C"
