// FP8 (E4M3fn) block-128 quantisers, gfx950: activation rows, expert weights in
// both orders, and the weighted SwiGLU.  The block's scale is s = amax / 448 in
// FP32 and a code is E4M3(448 x / amax), nearest with ties to even.  All three are
// bound by memory: a bf16 element moves 3 bytes in and out, an FP32 one 5.
//
// A 16-lane group owns one block of 128 elements, 8 per lane, so the block's
// maximum is four shuffles away and every load and store instruction of a
// group covers whole 64-byte pieces of its row.  A workgroup takes 16 rows, so
// that the 16 scales of a block column leave as one 64-byte run of the
// [blocks][rows] scale array, the order in which the GEMM's row tiles read them.
//
// Measured (a copy runs at 5.1 TB/s): bf16 rows 32768 x 1536 in 29 us (5.3 TB/s), FP32
// rows 8192 x 8192 in 88 us (3.9), 32771 x 784 in 33 us (3.9; five bytes an element and
// rounding to odd, both near their limits); 128 weights of 1536 x 2048 in both orders in
// 302 us (5.3).  One token takes 3 to 4 us of the device, the launch.
#include "common.h"
#include "fp8.h"

namespace nvfp4moe {
namespace q8 {

constexpr int kRows = 16;          // rows per workgroup, one per 16-lane group
constexpr int kThreads = 256;
constexpr int64_t kMaxRows = (int64_t(1) << 28) - kRows;   // a launch holds fewer than 2^32 threads in x
constexpr float kMax = 448.0f;     // largest E4M3fn value

// amax of a 16-lane group
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
  return v;
}

// The quotients 448 x / amax that the codes are rounded from.  E4M3 keeps four bits,
// so a code is the nearest one if the float handed to the conversion lies on the
// right side of every midpoint, and on it for a tie.  For 2^-80 <= amax <= 2^80 the
// quotient is a product by y = fl(1 / amax) and one corrected step (Markstein), which
// rounds X / amax as one IEEE division does, X = fl(448 x):
// - a bf16 x makes X exact, and a quotient of 8-bit numbers that is not a midpoint is
//   2^-13 or more of itself away from one, so the rounded quotient decides;
// - an FP32 x (ODD) leaves X a tail `lo`, and its quotient can come within 2^-30 of a
//   midpoint: with e the sign of what the rounded quotient leaves, it is rounded to odd
//   (towards zero, the last bit set if inexact), which no midpoint is.
// A SwiGLU's FP32 h is itself rounded and takes the plain quotient.  Outside the range
// (and for an infinite amax) the division is one in float64, rounded to odd as well.
struct Ratio {
  float a, y;
  bool fast, zero;
  __device__ __forceinline__ Ratio(float amax, float s) : a(amax), zero(s == 0.0f) {
    fast = amax >= 0x1p-80f && amax <= 0x1p80f;
    y = 1.0f / (fast ? amax : 1.0f);
  }
  // q > 0 nearest to a quotient that is larger by something of e's sign -> rounded to odd
  static __device__ __forceinline__ float odd(float q, float e) {
    const int ei = __float_as_int(e);
    return __int_as_float((__float_as_int(q) + (ei >> 31)) | (int)min((uint32_t)ei, 1u));
  }
  // a NaN stays one; s == 0 gives 0
  template <bool ODD>
  __device__ __forceinline__ float of(float x) const {
    if (fast) {
      const float m = __builtin_fabsf(x), X = m * kMax;
      float q = X * y;
      if constexpr (ODD) {
        const float lo = __builtin_fmaf(m, kMax, -X);
        q = __builtin_fmaf(__builtin_fmaf(-q, a, X) + lo, y, q);
        q = odd(q, __builtin_fmaf(-q, a, X) + lo);
      } else {
        q = __builtin_fmaf(__builtin_fmaf(-q, a, X), y, q);
      }
      return __builtin_copysignf(q, x);   // on magnitudes: the corrected step makes a -0 positive
    }
    if (x != x) return x;
    if (zero) return 0.0f;
    const double t = (double)kMax * (double)__builtin_fabsf(x) / (double)a;
    const float q = (float)t;
    const double e = t - (double)q;
    return t != t ? (float)t : __builtin_copysignf(odd(q, e > 0.0 ? 1.0f : e < 0.0 ? -1.0f : 0.0f), x);
  }
};

// four quotients -> four E4M3 codes in one word
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ void unpack8(const uint4 w, float (&v)[8]) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

// Eight elements of a block per lane, in one of two placements (l = lane of the
// group): bf16 takes elements 8l .. 8l+7 (one 16-byte load), FP32 takes
// 4l .. 4l+3 and 64 + 4l .. +3 (two 16-byte loads), so each load of the group
// is contiguous.  `left` is the number of elements from the block's start to
// the row's end (a multiple of 16); elements past it are 0.
template <bool F32>
__device__ __forceinline__ void load_block(const void* base, int64_t at, int l, int left, float (&v)[8]) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(base) + at;
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = 4 * l < left ? *reinterpret_cast<const float4*>(p + 4 * l) : z;
    const float4 b = 64 + 4 * l < left ? *reinterpret_cast<const float4*>(p + 64 + 4 * l) : z;
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    unpack8(8 * l < left ? *reinterpret_cast<const uint4*>(p + 8 * l) : make_uint4(0, 0, 0, 0), v);
  }
}

// the block's codes at `out`, in the same placement
template <bool F32, bool ODD>
__device__ __forceinline__ void store_codes(uint8_t* out, int l, int left, const float (&v)[8], const Ratio& d) {
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = d.of<ODD>(v[j]);
  const uint32_t w0 = codes4(q[0], q[1], q[2], q[3]), w1 = codes4(q[4], q[5], q[6], q[7]);
  if constexpr (F32) {
    if (4 * l < left) *reinterpret_cast<uint32_t*>(out + 4 * l) = w0;
    if (64 + 4 * l < left) *reinterpret_cast<uint32_t*>(out + 64 + 4 * l) = w1;
  } else {
    if (8 * l < left) *reinterpret_cast<uint2*>(out + 8 * l) = make_uint2(w0, w1);
  }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, __builtin_fabsf(v[j]));
  return m;
}

// Workgroup (row group, block group): 16 rows x NB blocks, every load issued
// before the first maximum is formed.
template <bool F32, int NB>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(
    const void* __restrict__ x, int64_t rows, int K, const int32_t* __restrict__ offsets, int E,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int l = threadIdx.x & 15;
  const int64_t r = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 4);
  const int64_t live = offsets ? min(rows, (int64_t)offsets[E]) : rows;
  if (r >= live) return;
  const int k0 = (int)blockIdx.y * NB * kFp8Block;
  float v[NB][8];
#pragma unroll
  for (int b = 0; b < NB; ++b) load_block<F32>(x, r * K + k0 + b * kFp8Block, l, K - k0 - b * kFp8Block, v[b]);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int k = k0 + b * kFp8Block;
    if (k >= K) break;
    const float m = group_max(amax8(v[b])), s = m / kMax;
    store_codes<F32, F32>(codes + r * K + k, l, K - k, v[b], Ratio(m, s));
    if (l == 0) scales[(int64_t)(k / kFp8Block) * rows + r] = s;
  }
}

// g sigmoid(g) in FP32: with z = exp(-|g|) in (0, 1], sigmoid(g) is 1 / (1 + z)
// for g >= 0 and z / (1 + z) below, so nothing overflows and sigmoid(-inf) is 0
// (an infinite negative gate gives NaN, as g / (1 + exp(-g)) does).  exp is the
// hardware exp2 of |g| log2(e) split into a head and a tail (the product's
// rounding error would otherwise cost |g| 2^-24); the hardware flushes results
// below 2^-126, so there z is taken 2^64 times too large and the power is
// taken off the product.  The reciprocal is the hardware's with one Newton step.
// Within 2^-21 relative, and 2^-149 absolute where the result is subnormal.
__device__ __forceinline__ float silu(float g) {
  const float a = -__builtin_fabsf(g);
  const float t = a * 0x1.715476p+0f;
  const float lo = __builtin_fmaf(a, 0x1.4ae0cp-26f, __builtin_fmaf(a, 0x1.715476p+0f, -t));
  const bool tiny = a < -80.0f;
  float z = __builtin_amdgcn_exp2f(tiny ? t + 64.0f : t);
  z = a > -0x1p8f ? __builtin_fmaf(z, lo * 0x1.62e43p-1f, z) : z;   // not for an infinite g
  const float d = tiny ? 1.0f : 1.0f + z;
  float y = __builtin_amdgcn_rcpf(d);
  y = __builtin_fmaf(y, __builtin_fmaf(-d, y, 1.0f), y);
  return g >= 0.0f ? g * y : g * (z * y) * (tiny ? 0x1p-64f : 1.0f);
}

// One block per lane (two are no faster: 39 to 41 us either way for 32768 rows of 768 in
// bf16 with h kept, 177 MB at 4.5 TB/s; a copy of these bytes takes 35).
template <bool F32>
__global__ __launch_bounds__(kThreads) void swiglu_quantize_kernel(
    const void* __restrict__ gu, int64_t R_cap, int I, const int32_t* __restrict__ offsets, int E,
    const float* __restrict__ topk_w, const int32_t* __restrict__ row_to_tk,
    uint8_t* __restrict__ codes, float* __restrict__ scales, uint16_t* __restrict__ h_out) {
  const int l = threadIdx.x & 15;
  const int64_t r = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 4);
  if (r >= R_cap || r >= offsets[E]) return;
  const int k = (int)blockIdx.y * kFp8Block, left = I - k;
  float g[8], u[8];
  load_block<F32>(gu, r * 2 * I + k, l, left, g);
  load_block<F32>(gu, r * 2 * I + I + k, l, left, u);
  float w = 1.0f;
  if (topk_w) {   // the router weight of the row's (token, slot); a bad map entry gives 0
    const int32_t i = row_to_tk[r];
    w = (i >= 0 && i < R_cap) ? topk_w[i] : 0.0f;
  }
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[j] = silu(g[j]) * u[j];
    if (topk_w) h[j] *= w;
  }
  const float m = group_max(amax8(h)), s = m / kMax;
  store_codes<F32, false>(codes + r * I + k, l, left, h, Ratio(m, s));
  if (l == 0) scales[(int64_t)(k / kFp8Block) * R_cap + r] = s;
  if (h_out) {
    uint16_t* p = h_out + r * I + k;
    if constexpr (F32) {
      if (4 * l < left) *reinterpret_cast<uint2*>(p + 4 * l) = make_uint2(bf16x2_rne(h[0], h[1]), bf16x2_rne(h[2], h[3]));
      if (64 + 4 * l < left) *reinterpret_cast<uint2*>(p + 64 + 4 * l) = make_uint2(bf16x2_rne(h[4], h[5]), bf16x2_rne(h[6], h[7]));
    } else if (8 * l < left) {
      *reinterpret_cast<uint4*>(p + 8 * l) = make_uint4(bf16x2_rne(h[0], h[1]), bf16x2_rne(h[2], h[3]),
                                                        bf16x2_rne(h[4], h[5]), bf16x2_rne(h[6], h[7]));
    }
  }
}

// One 128 x 128 block of a weight matrix per workgroup.  Thread t holds the
// 8 x 8 elements of rows 8 (t / 16) .. +7 and columns 8 (t % 16) .. +7; the
// maximum goes over the workgroup through LDS.  Its rows are stored as they
// lie.  The transposed codes come from converting the same registers in pairs
// down the rows, so no byte is moved for it: each thread has, per column, the
// 8 codes of its 8 rows, and the block crosses LDS only to leave as 16-byte
// pieces of whole 128-byte rows of the transposed matrix.
__global__ __launch_bounds__(kThreads) void quantize_weights_kernel(
    const uint16_t* __restrict__ w, int N, int K, uint8_t* __restrict__ codes,
    float* __restrict__ scales, uint8_t* __restrict__ codes_t, float* __restrict__ scales_t) {
  __shared__ float wmax[kThreads / kWave];
  __shared__ __align__(16) uint8_t tile[kFp8Block * kFp8Block];
  const int tid = threadIdx.x, ng = tid >> 4, kg = tid & 15;
  const int kb = blockIdx.x, nb = blockIdx.y;
  const int64_t e = blockIdx.z;
  const int n0 = nb * kFp8Block + 8 * ng, k0 = kb * kFp8Block + 8 * kg;
  const uint16_t* src = w + (e * N + n0) * K + k0;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    unpack8(n0 + i < N && k0 < K ? *reinterpret_cast<const uint4*>(src + (int64_t)i * K) : make_uint4(0, 0, 0, 0), v[i]);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
  m = wave_max(m);
  if ((tid & (kWave - 1)) == 0) wmax[tid / kWave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
  const float s = m / kMax;
  const Ratio d(m, s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = d.of<false>(v[i][j]);
  const int nn = (N + kFp8Block - 1) / kFp8Block, nk = (K + kFp8Block - 1) / kFp8Block;
  if (codes) {
    uint8_t* dst = codes + (e * N + n0) * K + k0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n0 + i < N && k0 < K)
        *reinterpret_cast<uint2*>(dst + (int64_t)i * K) =
            make_uint2(codes4(v[i][0], v[i][1], v[i][2], v[i][3]), codes4(v[i][4], v[i][5], v[i][6], v[i][7]));
    if (tid == 0) scales[(e * nn + nb) * nk + kb] = s;
  }
  if (codes_t) {
    // row k of the tile holds 16 pieces of 8 bytes, piece p at p ^ (k / 8): the
    // 16 lanes that write one k / 8 apart land on different banks
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<uint2*>(tile + (8 * kg + j) * kFp8Block + 8 * (ng ^ kg)) =
          make_uint2(codes4(v[0][j], v[1][j], v[2][j], v[3][j]), codes4(v[4][j], v[5][j], v[6][j], v[7][j]));
    __syncthreads();
    uint8_t* dst = codes_t + e * N * K;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = 32 * u + (tid >> 3), c = tid & 7;          // 16-byte piece c of tile row k
      const int k = kb * kFp8Block + row, n = nb * kFp8Block + 16 * c;
      const uint2 a = *reinterpret_cast<const uint2*>(tile + row * kFp8Block + 8 * ((2 * c) ^ (row >> 3)));
      const uint2 b = *reinterpret_cast<const uint2*>(tile + row * kFp8Block + 8 * ((2 * c + 1) ^ (row >> 3)));
      if (k < K && n < N) *reinterpret_cast<uint4*>(dst + (int64_t)k * N + n) = make_uint4(a.x, a.y, b.x, b.y);
    }
    if (tid == 0) scales_t[(e * nk + kb) * nn + nb] = s;
  }
}

// Blocks from which a row quantiser's lane takes four: with one, 65536 blocks of FP32 take
// 11.5 us (four: 13.9) and 262144 of bf16 19.8 (21.8), while 393216 of bf16 take 34 (29)
// and 524288 of FP32 101 (88).
constexpr int64_t kLongBlocks = 327680;

}  // namespace q8
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

NVFP4MOE_API int fp8_quantize_rows(const void* x, int32_t x_dtype, int64_t rows, int64_t K,
                                   const int32_t* expert_offsets, int32_t E, uint8_t* codes,
                                   float* scales, void* stream) {
  if (x_dtype != NVFP4_IN_BF16 && x_dtype != NVFP4_IN_F32) return NVFP4_ERR_ARG;
  if (rows < 0 || rows > q8::kMaxRows || K <= 0 || K % 16 != 0 || K > FP8_MAX_K) return NVFP4_ERR_SHAPE;
  if (expert_offsets && (E < 1 || E > NVFP4MOE_MAX_EXPERTS)) return NVFP4_ERR_SHAPE;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return NVFP4_ERR_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t nk = (K + kFp8Block - 1) / kFp8Block;
  const int nb = rows * nk >= q8::kLongBlocks ? 4 : 1;
  const dim3 grid((unsigned)((rows + q8::kRows - 1) / q8::kRows), (unsigned)((nk + nb - 1) / nb));
#define FP8_ROWS(F32, NB) \
  q8::quantize_rows_kernel<F32, NB><<<grid, q8::kThreads, 0, s>>>(x, rows, (int)K, expert_offsets, E, codes, scales)
  if (x_dtype == NVFP4_IN_F32) {
    if (nb == 4) FP8_ROWS(true, 4); else FP8_ROWS(true, 1);
  } else {
    if (nb == 4) FP8_ROWS(false, 4); else FP8_ROWS(false, 1);
  }
#undef FP8_ROWS
  return launch_status();
}

NVFP4MOE_API int fp8_swiglu_quantize(const void* gu, int32_t gu_dtype, int64_t R_cap, int64_t I,
                                     const int32_t* expert_offsets, int32_t E, const float* topk_w,
                                     const int32_t* row_to_tk, uint8_t* codes, float* scales,
                                     uint16_t* h_out, void* stream) {
  if (gu_dtype != NVFP4_IN_BF16 && gu_dtype != NVFP4_IN_F32) return NVFP4_ERR_ARG;
  if (R_cap < 0 || R_cap > q8::kMaxRows || I <= 0 || I % 16 != 0 || I > FP8_MAX_K) return NVFP4_ERR_SHAPE;
  if (E < 1 || E > NVFP4MOE_MAX_EXPERTS) return NVFP4_ERR_SHAPE;
  if (R_cap == 0) return NVFP4_OK;
  if (!gu || !expert_offsets || !codes || !scales || (topk_w && !row_to_tk)) return NVFP4_ERR_NULL;
  if (!aligned16(gu) || !aligned16(codes) || !aligned16(scales) || !aligned16(h_out)) return NVFP4_ERR_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)((R_cap + q8::kRows - 1) / q8::kRows), (unsigned)((I + kFp8Block - 1) / kFp8Block));
#define FP8_SWIGLU(F32) \
  q8::swiglu_quantize_kernel<F32><<<grid, q8::kThreads, 0, s>>>(gu, R_cap, (int)I, expert_offsets, E, topk_w, row_to_tk, codes, scales, h_out)
  if (gu_dtype == NVFP4_IN_F32) FP8_SWIGLU(true);
  else FP8_SWIGLU(false);
#undef FP8_SWIGLU
  return launch_status();
}

NVFP4MOE_API int fp8_quantize_weights(const uint16_t* w, int64_t E, int64_t N, int64_t K, uint8_t* codes,
                                      float* scales, uint8_t* codes_t, float* scales_t, void* stream) {
  if (E < 0 || E > 65535 || N < 1 || N > FP8_MAX_N || K <= 0 || K % 16 != 0 || K > FP8_MAX_K) return NVFP4_ERR_SHAPE;
  if (codes_t && (N % 16 != 0 || N > FP8_MAX_K)) return NVFP4_ERR_SHAPE;
  if (E == 0) return NVFP4_OK;
  if (!w || (!codes && !codes_t) || (codes && !scales) || (codes_t && !scales_t)) return NVFP4_ERR_NULL;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales) || !aligned16(codes_t) || !aligned16(scales_t))
    return NVFP4_ERR_ALIGN;
  const dim3 grid((unsigned)((K + kFp8Block - 1) / kFp8Block), (unsigned)((N + kFp8Block - 1) / kFp8Block), (unsigned)E);
  q8::quantize_weights_kernel<<<grid, q8::kThreads, 0, static_cast<hipStream_t>(stream)>>>(
      w, (int)N, (int)K, codes, scales, codes_t, scales_t);
  return launch_status();
}

}  // extern "C"
