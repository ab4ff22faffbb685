// Token rows sorted by expert without quantising them, the weighted way back to token order, and its
// gradient, for gfx950.  All are bound by memory: the sort reads every token row once and writes it k
// times, the combine reads k rows for each that it writes, the gradient reads and writes k rows a token.
#include "common.h"
#include "route.h"
#include "rows.h"

namespace nvfp4moe {
namespace mp {

constexpr int kWaves = 4;       // wavefronts per 256-thread workgroup
constexpr int kCols = 512;      // elements of a row that a wavefront takes at a time, 8 a lane

// One wavefront per token: its entries' rows from the first rows of route_scan_kernel, the maps, and the
// token's row (bytes, a multiple of 16) copied to them.
__global__ __launch_bounds__(kWaves * 64) void permute_rows_kernel(
    const uint4* __restrict__ x, int64_t T, int words, const int32_t* __restrict__ ids, int k, int E,
    const int32_t* __restrict__ base, const int32_t* __restrict__ rank, int chunk_log, uint4* __restrict__ rows,
    int32_t* __restrict__ row_to_tk, int32_t* __restrict__ tk_to_row) {
  const int64_t t = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= T) return;
  const int lane = lane_id();
  int row = -1;
  if (lane < k) {
    const int i = (int)(t * k) + lane;
    const int r = rank[i];
    if (r >= 0) row = base[(int64_t)(i >> chunk_log) * E + ids[i]] + r;
    tk_to_row[i] = row;
    if (row >= 0) row_to_tk[row] = i;
  }
  if (!rows) return;
  for (int c0 = 0; c0 < words; c0 += kWave) {
    const int c = c0 + lane;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < words) v = x[t * words + c];
    for (int s = 0; s < k; ++s) {
      const int r = __shfl(row, s, kWave);
      if (r >= 0 && c < words) rows[(int64_t)r * words + c] = v;
    }
  }
}

// One wavefront per 512 columns of a token's sum, taken in FP32 and in slot order with products and sums
// rounded apart; the loads of 8 slots are issued before the first is added.
template <bool DF32, bool YF32>
__global__ __launch_bounds__(kWaves * 64) void combine_kernel(
    const void* __restrict__ d, int64_t T, int k, int H, const int32_t* __restrict__ tk_to_row,
    const float* __restrict__ topk_w, void* __restrict__ y) {
  const int pieces = (H + kCols - 1) / kCols;
  const int64_t item = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int64_t t = item / pieces;
  if (t >= T) return;
  const int lane = lane_id();
  const int my_row = lane < k ? tk_to_row[t * k + lane] : -1;
  const float my_w = (lane < k && topk_w) ? topk_w[t * k + lane] : 1.0f;
  const int c = (int)(item - t * pieces) * kCols + 8 * lane;
  const bool inside = c < H;
  float acc[8] = {};
  bool started = false;
  for (int s0 = 0; s0 < k; s0 += 8) {
    Raw8<DF32> raw[8];
    bool ok[8];
    float ws[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int row = __shfl(my_row, s0 + u, kWave);   // s0 + u < 40: a lane; entries past k have no row
      ws[u] = __shfl(my_w, s0 + u, kWave);
      ok[u] = row >= 0 && row < T * k && inside;
      if (ok[u]) raw[u] = load8<DF32>(d, (int64_t)row * H + c);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (!ok[u]) continue;
      float v[8];
      unpack8<DF32>(raw[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = topk_w ? ws[u] * v[j] : v[j];
        acc[j] = started ? acc[j] + x : x;
      }
      started = true;
    }
  }
  if (inside) store8<YF32>(y, t * H + c, acc);
}

// One wavefront per entry i = (t, s): dd[row] = w_i dy[t], dw_i = <dy[t], d[row]> in FP32, added within
// the lane and then over the wavefront in a fixed order.  An entry without a row has dw_i = 0.
template <bool YF32, bool DF32>
__global__ __launch_bounds__(kWaves * 64) void combine_backward_kernel(
    const void* __restrict__ dy, const void* __restrict__ d, int64_t R, int k, int H,
    const int32_t* __restrict__ tk_to_row, const float* __restrict__ topk_w, void* __restrict__ dd,
    float* __restrict__ dw) {
  const int64_t i = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (i >= R) return;
  const int64_t row = tk_to_row[i];
  const bool has = row >= 0 && row < R;
  const int64_t t = i / k;
  const int lane = lane_id();
  float sum = 0.0f;
  if (has) {
    const float w = topk_w ? topk_w[i] : 1.0f;
    for (int c = 8 * lane; c < H; c += kCols) {
      float g[8], v[8];
      unpack8<YF32>(load8<YF32>(dy, t * H + c), g);
      if (dw) {
        unpack8<DF32>(load8<DF32>(d, row * H + c), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(g[j], v[j], sum);
      }
      if (dd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = w * g[j];
        store8<DF32>(dd, row * H + c, v);
      }
    }
  }
  if (dw) {
    sum = wave_sum(sum);
    if (lane == 0) dw[i] = sum;
  }
}

inline bool type_ok(int32_t t) { return t == NVFP4_IN_BF16 || t == NVFP4_IN_F32; }

inline int check(int64_t T, int32_t k, int64_t H) {
  if (T < 0 || k < 1 || k > NVFP4MOE_MAX_TOPK || H < 8 || H % 8 != 0 || H > MOE_MAX_H) return NVFP4_ERR_SHAPE;
  return T * (int64_t)k > INT32_MAX / 2 ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

}  // namespace mp
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

NVFP4MOE_API int moe_permute(const void* x, int32_t x_dtype, int64_t T, int64_t H, const int32_t* topk_ids, int32_t k,
                             int32_t E, void* rows, int32_t* expert_offsets, int32_t* row_to_tk, int32_t* tk_to_row,
                             void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  if (!mp::type_ok(x_dtype)) return NVFP4_ERR_ARG;
  if (const int bad = mp::check(T, k, x || rows ? H : 8)) return bad;
  if (E < 1 || E > NVFP4MOE_MAX_EXPERTS || k > E) return NVFP4_ERR_SHAPE;
  if (!expert_offsets || !workspace) return NVFP4_ERR_NULL;
  if (T > 0 && (!topk_ids || !row_to_tk || !tk_to_row || !x != !rows)) return NVFP4_ERR_NULL;
  if (!aligned16(x) || !aligned16(topk_ids) || !aligned16(rows) || !aligned16(expert_offsets) ||
      !aligned16(row_to_tk) || !aligned16(tk_to_row) || !aligned16(workspace))
    return NVFP4_ERR_ALIGN;
  if (x && x == rows) return NVFP4_ERR_ARG;
  if (workspace_bytes < nvfp4moe_permute_workspace_size(T, k, E)) return NVFP4_ERR_WORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n = T * (int64_t)k;
  const int chunk_log = plan_chunk_log(n, E), chunks = plan_chunks(n, chunk_log);
  int32_t* table = static_cast<int32_t*>(workspace);        // [chunks][E]
  int32_t* rank = table + (int64_t)chunks * E;              // [n]
  route_rank_kernel<<<chunks, kPlanThreads, 0, s>>>(topk_ids, (int)n, E, chunk_log, table, rank, dev_err);
  route_scan_kernel<<<1, kPlanThreads, 0, s>>>(table, chunks, E, expert_offsets);
  if (T > 0) {
    const int words = (int)(H * (x_dtype == NVFP4_IN_F32 ? 4 : 2) / 16);
    mp::permute_rows_kernel<<<(unsigned)((T + mp::kWaves - 1) / mp::kWaves), mp::kWaves * 64, 0, s>>>(
        static_cast<const uint4*>(x), T, words, topk_ids, k, E, table, rank, chunk_log, static_cast<uint4*>(rows),
        row_to_tk, tk_to_row);
  }
  return launch_status();
}

NVFP4MOE_API int moe_combine(const void* d, int32_t d_dtype, int64_t T, int32_t k, int64_t H, const int32_t* tk_to_row,
                             const float* topk_w, void* y, int32_t y_dtype, void* stream) {
  if (!mp::type_ok(d_dtype) || !mp::type_ok(y_dtype)) return NVFP4_ERR_ARG;
  if (const int bad = mp::check(T, k, H)) return bad;
  if (T == 0) return NVFP4_OK;
  if (!d || !tk_to_row || !y) return NVFP4_ERR_NULL;
  if (!aligned16(d) || !aligned16(tk_to_row) || !aligned16(topk_w) || !aligned16(y)) return NVFP4_ERR_ALIGN;
  if (d == y) return NVFP4_ERR_ARG;
  const int64_t items = T * ((H + mp::kCols - 1) / mp::kCols);
  const int64_t grid = (items + mp::kWaves - 1) / mp::kWaves;
  if (grid > INT32_MAX) return NVFP4_ERR_SHAPE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool df = d_dtype == NVFP4_IN_F32, yf = y_dtype == NVFP4_IN_F32;
#define MP_COMBINE(D, Y) mp::combine_kernel<D, Y><<<(unsigned)grid, mp::kWaves * 64, 0, s>>>(d, T, k, (int)H, tk_to_row, topk_w, y)
  if (df) yf ? MP_COMBINE(true, true) : MP_COMBINE(true, false);
  else yf ? MP_COMBINE(false, true) : MP_COMBINE(false, false);
#undef MP_COMBINE
  return launch_status();
}

NVFP4MOE_API int moe_combine_backward(const void* dy, int32_t dy_dtype, const void* d, int32_t d_dtype, int64_t T,
                                      int32_t k, int64_t H, const int32_t* tk_to_row, const float* topk_w, void* dd,
                                      float* dtopk_w, void* stream) {
  if (!mp::type_ok(dy_dtype) || !mp::type_ok(d_dtype)) return NVFP4_ERR_ARG;
  if (const int bad = mp::check(T, k, H)) return bad;
  if (T == 0) return NVFP4_OK;
  if (!dy || !tk_to_row || (!dd && !dtopk_w) || (dtopk_w && !d)) return NVFP4_ERR_NULL;
  if (!aligned16(dy) || !aligned16(d) || !aligned16(tk_to_row) || !aligned16(topk_w) || !aligned16(dd) ||
      !aligned16(dtopk_w))
    return NVFP4_ERR_ALIGN;
  if (dd && (dd == d || dd == dy)) return NVFP4_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t R = T * (int64_t)k;
  const unsigned grid = (unsigned)((R + mp::kWaves - 1) / mp::kWaves);
  const bool yf = dy_dtype == NVFP4_IN_F32, df = d_dtype == NVFP4_IN_F32;
#define MP_BACKWARD(Y, D) \
  mp::combine_backward_kernel<Y, D><<<grid, mp::kWaves * 64, 0, s>>>(dy, d, R, k, (int)H, tk_to_row, topk_w, dd, dtopk_w)
  if (yf) df ? MP_BACKWARD(true, true) : MP_BACKWARD(true, false);
  else df ? MP_BACKWARD(false, true) : MP_BACKWARD(false, false);
#undef MP_BACKWARD
  return launch_status();
}

}  // extern "C"
