// Token rows sorted by expert without quantising them, the weighted way back to token order, and its
// gradient, for gfx950.  All are bound by memory: the sort reads every token row once and writes it k
// times, the combine reads k rows for each that it writes, the gradient reads and writes k rows a token.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "route.h"
#include "rows.h"

namespace nvfp4moe {
namespace mp {

constexpr int kThreads = 256;

// Rows go out with non-temporal stores: 4096 tokens x 8 rows of 4 KB take 27 us so and 36 with ordinary
// ones (in both cases after other work has left the caches full of lines to write back).  The grouped
// product that reads them next gains less from their being cached than that: permutation and a BF16 gate_up
// product together take 169 us for 176 at 600 tokens, 202 for 201 at 2048, 247 for 249 at 4096, 361 for 381
// at 8192.  Short rows gain or lose little: 16384 tokens x 8 rows of 16 bytes 18.4 us for 18.0, of 64 17.6 for
// 17.8, of 128 18.3 for 19.1, of 512 25.1 for 24.5, of 1024 37.8 for 41.8 (with a combine of the rows next 25.3
// for 25.4, 22.6 for 23.8, 24.7 for 24.8, 40.4 for 37.6 and 64.7 for 59.1).
__device__ __forceinline__ void store_row(uint4* dst, uint4 v) { store16<true>(dst, v); }

// A wavefront's part of a token's row: its first kHeld 16-byte words a lane stay in registers (rows up to
// 4 KB), requested before the routing is known; longer rows are read again for what lies behind.
constexpr int kHeld = 4;
struct Row {
  uint4 held[kHeld];
  __device__ __forceinline__ void load(const uint4* __restrict__ src, int words) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u) held[u] = src[min(u * kWave + lane_id(), words - 1)];
  }
  __device__ __forceinline__ void load(const uint4* __restrict__ src, int words, int group) {
    if (group < kWave) held[0] = src[min(lane_id() & (group - 1), words - 1)];
    else load(src, words);
  }
  __device__ __forceinline__ void copy_held(uint4* __restrict__ dst, int words) const {
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (u * kWave + lane_id() < words) store_row(dst + u * kWave + lane_id(), held[u]);
  }
};

// The token's row to its k routed rows (row: lane s holds entry s's, -1 for none).  Rows of at most 32 words
// (held repeated over the wavefront) go out several at a time.
__device__ __forceinline__ void copy_to_rows(const Row& held, const uint4* __restrict__ src, int words, int group, int k,
                                             int row, uint4* __restrict__ rows) {
  if (group < kWave) {
    const int c = lane_id() & (group - 1);
    for (int s0 = 0; s0 < k; s0 += kWave / group) {
      const int s = s0 + lane_id() / group;        // < 96
      const int r = __shfl(row, s & (kWave - 1), kWave);
      if (s < k && r >= 0 && c < words) store_row(rows + (int64_t)r * words + c, held.held[0]);
    }
    return;
  }
  for (int s = 0; s < k; ++s) {
    const int r = __shfl(row, s, kWave);
    if (r >= 0) held.copy_held(rows + (int64_t)r * words, words);
  }
  for (int c0 = kHeld * kWave; c0 < words; c0 += kWave) {
    const int c = c0 + lane_id();
    const uint4 v = src[min(c, words - 1)];
    for (int s = 0; s < k; ++s) {
      const int r = __shfl(row, s, kWave);
      if (r >= 0 && c < words) store_row(rows + (int64_t)r * words + c, v);
    }
  }
}

// Long routing lists, whose count table no workgroup could scan: one wavefront-wide column of 64 experts per
// workgroup, its 16 wavefronts a part of the chunks each.  table[c][e] becomes the entries of e in the chunks
// before c, total[e] those of all.  (508000 entries of 1000 experts, the maps alone: 25 us, 65 with one workgroup
// that scans the whole table.)
constexpr int kColumnWaves = 16;
__global__ __launch_bounds__(kColumnWaves * 64) void route_columns_kernel(int32_t* __restrict__ table, int nchunks, int E,
                                                                          int32_t* __restrict__ total) {
  __shared__ int32_t part[kColumnWaves][kWave];
  const int lane = lane_id(), wave = threadIdx.x >> 6, e = blockIdx.x * kWave + lane;
  const int per = (nchunks + kColumnWaves - 1) / kColumnWaves;
  const int lo = min(nchunks, wave * per), hi = min(nchunks, lo + per);
  int sum = 0;
  if (e < E)
    for (int c = lo; c < hi; ++c) sum += table[(int64_t)c * E + e];
  part[wave][lane] = sum;
  __syncthreads();
  if (e >= E) return;
  int acc = 0;
  for (int w = 0; w < wave; ++w) acc += part[w][lane];
  if (wave == kColumnWaves - 1) total[e] = acc + sum;
  for (int c = lo; c < hi; ++c) {
    const int64_t at = (int64_t)c * E + e;
    const int v = table[at];
    table[at] = acc;
    acc += v;
  }
}

// The expert offsets from the experts' totals, into LDS (and memory, from workgroup 0).
__device__ __forceinline__ void scan_totals(const int32_t* total, int E, int32_t* first, int32_t* wsum,
                                            int32_t* __restrict__ offsets) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  int tot[kRouteExp], sum = 0;
#pragma unroll
  for (int u = 0; u < kRouteExp; ++u) {
    const int e = kRouteExp * tid + u;
    tot[u] = e < E ? total[e] : 0;
    sum += tot[u];
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int y = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += y;
  }
  if (lane == kWave - 1) wsum[wave] = incl;
  __syncthreads();
  int at = incl - sum;
  for (int w = 0; w < wave; ++w) at += wsum[w];
#pragma unroll
  for (int u = 0; u < kRouteExp; ++u) {
    const int e = kRouteExp * tid + u;
    if (e < E) {
      first[e] = at;
      if (blockIdx.x == 0) offsets[e] = at;
    }
    at += tot[u];
  }
  if (blockIdx.x == 0 && tid == kRouteThreads - 1) offsets[E] = at;
  __syncthreads();
}

// The main pass: `rounds` tokens to each of a workgroup's eight wavefronts, the entries' rows from their ranks
// and from the count table (TABLE) or the columns' sums, the maps, and the token's row copied to them.  The
// first token's row is requested before the table is scanned, each later one before the copies of the token
// ahead of it.  4096 tokens x 8 rows of 2048 bf16: 28 us, 152 MB at 5.4 TB/s; without the scan, at made-up rows,
// 26 to 28, so it is hidden.
struct TotalsLds {
  int32_t first[NVFP4MOE_MAX_EXPERTS], wsum[kRouteWaves];
};
template <bool TABLE>
__global__ __launch_bounds__(kRouteThreads) void permute_kernel(
    const uint4* __restrict__ x, int64_t T, int words, const int32_t* __restrict__ ids, int k, int E,
    const int32_t* __restrict__ cnt, const int32_t* __restrict__ rank, const int32_t* __restrict__ total, int nchunks,
    int chunk_log, int rounds, int group, uint4* __restrict__ rows, int32_t* __restrict__ offsets,
    int32_t* __restrict__ row_to_tk, int32_t* __restrict__ tk_to_row) {
  __shared__ std::conditional_t<TABLE, RouteLds, TotalsLds> lds;
  const int lane = lane_id();
  const int64_t t0 = (int64_t)blockIdx.x * kRouteTokens * rounds;   // the workgroup's first token
  int64_t t = t0 + (threadIdx.x >> 6);
  const int n = (int)(T * k);
  RouteTable table;
  if constexpr (TABLE) {
    table.c0 = (int)(t0 * k) >> chunk_log;
    table.load(cnt, nchunks * E);
  }
  int i = (int)(min(t, T - 1) * k) + lane;
  int e = ids[min(i, n - 1)], r = rank[min(i, n - 1)];
  Row held;
  if (rows) held.load(x + min(t, T - 1) * words, words, group);
  if constexpr (TABLE) table.scan(lds, nchunks, E, offsets);
  else scan_totals(total, E, lds.first, lds.wsum, offsets);
  for (int u = 0; u < rounds && t < T; ++u) {
    int row = -1;
    if (lane < k) {
      if (r >= 0) {                                // a rank marks a valid expert id
        if constexpr (TABLE) row = lds.first[(i >> chunk_log) - table.c0][e] + r;
        else row = lds.first[e] + cnt[(int64_t)(i >> chunk_log) * E + e] + r;
      }
      tk_to_row[i] = row;
      if (row >= 0) row_to_tk[row] = i;
    }
    const int64_t next = t + kRouteTokens;
    const uint4* src = x + t * words;
    Row ahead = held;
    i = (int)(min(next, T - 1) * k) + lane;
    if (u + 1 < rounds) {
      e = ids[min(i, n - 1)];
      r = rank[min(i, n - 1)];
      if (rows) ahead.load(x + min(next, T - 1) * words, words, group);
    }
    if (rows) copy_to_rows(held, src, words, group, k, row, rows);
    held = ahead;
    t = next;
  }
}

// Short routing lists in one launch: every workgroup reads the whole list, counts each expert's entries and
// those before its own (LDS; sums of whole numbers, whose order changes nothing), scans the counts, and ranks
// the entries of its own `per` tokens; its wavefronts then take one (token, slot) row each.
//
// The border was measured at 128 experts and 8 slots, with rows of 4 KB (3200 entries in one launch and in two 7.2 us
// for 9.8, 6144 10.0 for 10.8, 8192 12.2 for 12.2, 16384 21.9 for 19.2).  At 6144 entries, the maps alone, one
// launch takes 7.1 to 7.3 us for 8.0 to 9.9 with 8 slots of 8 to 1024 experts, 7.9 for 9.8 with one slot of 128, 8.4
// for 9.6 of 32; with one slot of 8 experts 10.9 for 9.3 and of 2 19.7 for 9.1 (two slots 13.2 for 8.4), because all
// lanes add to the same few counters and more workgroups read the list: there two launches are faster from 5000 and
// from 2500 entries on.
constexpr int kShort = 6144;            // entries
constexpr int kShortTokens = 8;         // most tokens a workgroup
__global__ __launch_bounds__(kRouteThreads) void permute_short_kernel(
    const uint4* __restrict__ x, int T, int words, const int32_t* __restrict__ ids, int k, int E, int per,
    uint4* __restrict__ rows, int32_t* __restrict__ offsets, int32_t* __restrict__ row_to_tk,
    int32_t* __restrict__ tk_to_row, int32_t* __restrict__ dev_err) {
  __shared__ int32_t total[NVFP4MOE_MAX_EXPERTS], before[NVFP4MOE_MAX_EXPERTS], first[NVFP4MOE_MAX_EXPERTS];
  __shared__ int32_t own_e[kShortTokens * NVFP4MOE_MAX_TOPK], own_row[kShortTokens * NVFP4MOE_MAX_TOPK];
  __shared__ int32_t wsum[kRouteWaves];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int n = T * k, t0 = blockIdx.x * per, e0 = t0 * k, own = min(per, T - t0) * k;
  for (int e = tid; e < E; e += kRouteThreads) total[e] = before[e] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < n; i += kRouteThreads) {
    const int e = ids[i];
    const bool valid = e >= 0 && e < E;
    if (valid) {
      atomicAdd(&total[e], 1);
      if (i < e0) atomicAdd(&before[e], 1);
    }
    bad |= !valid;
    if (i >= e0 && i < e0 + own) own_e[i - e0] = valid ? e : -1;
  }
  if (bad && dev_err && blockIdx.x == 0) atomicOr(dev_err, NVFP4_DEVERR_BAD_EXPERT);
  __syncthreads();
  scan_totals(total, E, first, wsum, offsets);
  if (tid < own) {
    const int e = own_e[tid];
    int row = -1;
    if (e >= 0) {
      row = first[e] + before[e];
      for (int j = 0; j < tid; ++j) row += own_e[j] == e;
      row_to_tk[row] = e0 + tid;
    }
    tk_to_row[e0 + tid] = row;
    own_row[tid] = row;
  }
  if (!rows) return;
  __syncthreads();
  for (int q = wave; q < own; q += kRouteWaves) {
    const int row = own_row[q];
    if (row < 0) continue;
    const uint4* src = x + (int64_t)(t0 + q / k) * words;
    uint4* dst = rows + (int64_t)row * words;
    for (int c0 = 0; c0 < words; c0 += kHeld * kWave) {
      Row r;
      r.load(src + c0, words - c0);
      r.copy_held(dst + c0, words - c0);
    }
  }
}

// One lane per 8 columns of a token's sum, taken in FP32 and in slot order with products and sums rounded apart;
// the loads of 8 slots are issued before the first is added.  They are non-temporal: each row is read once (4096
// tokens x 8 rows of 2048 bf16: 27 us for 29; 151 MB, so 5.6 TB/s).  Every lane reads the token's rows and
// weights itself (handed round a wavefront with shuffles they take 26.2 us for 26.5 there, 36.9 for 34.4 at
// 16384 tokens with 2 rows), so that a wavefront may go over from one token to the next and no lane is without
// columns, whatever the row's length (16384 tokens x 8 rows of 520 bf16: 30 us, 34 with whole wavefronts a token).
// Of float32 rows to bf16, which unpermute_combine takes too and with the same bits: 61 tokens x 8 rows of 2048 4.9
// us, its kernels 8.6; 1024 15.5 and 14.8; 4096 58.9 and 54.4, of 768 25.9 and 19.1, of 7168 204 and 208; 16384 of
// 64 10.6 and 13.3, of 520 69 and 61.
template <bool DF32, bool YF32>
__global__ __launch_bounds__(kThreads) void combine_kernel(
    const void* __restrict__ d, int T, int k, int H, const int32_t* __restrict__ tk_to_row,
    const float* __restrict__ topk_w, void* __restrict__ y) {
  const uint32_t words = (uint32_t)H / 8, item = blockIdx.x * kThreads + threadIdx.x, t = item / words;
  if (t >= (uint32_t)T) return;
  const int c = (int)(item - t * words) * 8, R = T * k;
  const int32_t* map = tk_to_row + (int64_t)t * k;
  const float* wt = topk_w ? topk_w + (int64_t)t * k : nullptr;
  float acc[8] = {};
  bool started = false;
  for (int s0 = 0; s0 < k; s0 += 8) {
    Raw8<DF32> raw[8];
    int row[8];
    float ws[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      row[u] = s0 + u < k ? map[s0 + u] : -1;
      ws[u] = wt && s0 + u < k ? wt[s0 + u] : 1.0f;
      if (row[u] >= R) row[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (row[u] >= 0) raw[u] = load8<DF32, true>(d, (int64_t)row[u] * H + c);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (row[u] < 0) continue;
      float v[8];
      unpack8<DF32>(raw[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = wt ? ws[u] * v[j] : v[j];
        acc[j] = started ? acc[j] + x : x;
      }
      started = true;
    }
  }
  store8<YF32>(y, (int64_t)t * H + c, acc);
}

// Lanes that take an entry's row, a power of two: as many as hold it 8 elements a lane, up to a wavefront; half a
// wavefront for the rows just longer than that, of which a wavefront's second step would have few (16384 tokens
// x 8 rows of 64 bf16 7.8 us, with a wavefront a row 44.8; of 520, 61.8 and 79.5; but of 264 float32, which a
// wavefront holds, 72 us, 83 with 16 lanes).
constexpr int kAhead = 4;
inline int log_lanes_for(int64_t words) {
  if (words > 64) return words <= 96 ? 5 : 6;
  int lg = 0;
  while ((1 << lg) < words) ++lg;
  return lg;
}

// One group of 2^lg lanes per entry i = (t, s): dd[row] = w_i dy[t], dw_i = <dy[t], d[row]> in FP64, added within
// the lane and then over the group in a fixed order and rounded once (an FP32 sum's error grows with the row and
// shows where its terms cancel; it takes 58.4 us for 58.8 at 4096 tokens x 8 rows of 2048 bf16, 17.8 for 18.6 at
// 1024, of float32 124.7 both, one token 7 both).  An entry without a row has dw_i = 0.  The loads of AHEAD
// pieces of 8 * 2^lg columns are issued before the first is used (4096 tokens x 8 rows of 2048 bf16: 58 us
// with 4, 65 with 2, 70 with 1); a token's entries share dy[t] in the caches.  STREAM, where the operands do
// not fit the last-level cache: d and dd are non-temporal (54 us for 58; 285 MB, so 5.3 TB/s; with the BF16
// input-gradient product that reads dd next 256 us for 263, 377 for 390 at 8192 tokens, but 206 for 203 at
// 2048 and 166 for 162 at 512, where the caches hold them).
template <bool YF32, bool DF32, bool STREAM, int AHEAD>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const void* __restrict__ dy, const void* __restrict__ d, int R, int k, int H, int lg,
    const int32_t* __restrict__ tk_to_row, const float* __restrict__ topk_w, void* __restrict__ dd,
    float* __restrict__ dw) {
  const int i = (int)((blockIdx.x * kThreads + threadIdx.x) >> lg);
  const int lane = threadIdx.x & ((1 << lg) - 1), step = 8 << lg;
  const int64_t row = i < R ? tk_to_row[i] : -1;
  double sum = 0.0;
  if (row >= 0 && row < R) {
    const int64_t t = (uint32_t)i / (uint32_t)k;
    const float w = topk_w ? topk_w[i] : 1.0f;
    for (int c0 = 8 * lane; c0 < H; c0 += AHEAD * step) {
      Raw8<YF32> yr[AHEAD];
      Raw8<DF32> dr[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int c = min(c0 + u * step, H - 8);
        yr[u] = load8<YF32>(dy, t * H + c);
        if (dw) dr[u] = load8<DF32, STREAM>(d, row * H + c);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int c = c0 + u * step;
        if (c >= H) continue;
        float y[8], v[8];
        unpack8<YF32>(yr[u], y);
        if (dw) {
          unpack8<DF32>(dr[u], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)y[j], (double)v[j], sum);
        }
        if (dd) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = w * y[j];
          store8<DF32, STREAM>(dd, row * H + c, v);
        }
      }
    }
  }
  if (dw) {
    for (int off = 1 << lg >> 1; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, kWave);
    if (lane == 0 && i < R) dw[i] = (float)sum;
  }
}

constexpr int kChunkLog = kPlanChunkLogMin;

// Tokens a wavefront of the main pass takes: few enough workgroups that the table scans do not add up (131072
// entries, the maps alone: 13.5 us, 15.0 with one token each), a workgroup's entries in two chunks at most.
constexpr int kMainGroups = 1024;
inline int rounds_of(int64_t T, int k) {
  const int most = (1 << kChunkLog) / (kRouteTokens * k);
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, T / (kRouteTokens * kMainGroups)));
}

inline bool type_ok(int32_t t) { return t == NVFP4_IN_BF16 || t == NVFP4_IN_F32; }

inline int check(int64_t T, int32_t k, int64_t H) {
  if (T < 0 || k < 1 || k > NVFP4MOE_MAX_TOPK || H < 8 || H % 8 != 0 || H > MOE_MAX_H) return NVFP4_ERR_SHAPE;
  return T > MOE_MAX_ROWS || T * (int64_t)k > MOE_MAX_ROWS ? NVFP4_ERR_SHAPE : NVFP4_OK;
}

}  // namespace mp
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

NVFP4MOE_API size_t moe_permute_workspace_size(int64_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || k > NVFP4MOE_MAX_TOPK || E < 1 || E > NVFP4MOE_MAX_EXPERTS || T > MOE_MAX_ROWS) return 0;
  const int64_t n = T * (int64_t)k;
  if (T > 0 && n <= mp::kShort) return 0;
  // the (chunk, expert) count table, the experts' totals and a rank per entry
  const size_t bytes = ((size_t)plan_chunks(n, mp::kChunkLog) * E + E + (size_t)n) * sizeof(int32_t);
  return (bytes + 255) & ~(size_t)255;
}

NVFP4MOE_API int moe_permute(const void* x, int32_t x_dtype, int64_t T, int64_t H, const int32_t* topk_ids, int32_t k,
                             int32_t E, void* rows, int32_t* expert_offsets, int32_t* row_to_tk, int32_t* tk_to_row,
                             void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  if (!mp::type_ok(x_dtype)) return NVFP4_ERR_ARG;
  if (const int bad = mp::check(T, k, x || rows ? H : 8)) return bad;
  if (E < 1 || E > NVFP4MOE_MAX_EXPERTS || k > E) return NVFP4_ERR_SHAPE;
  const size_t need = T > 0 ? moe_permute_workspace_size(T, k, E) : 0;
  if (!expert_offsets || (need && !workspace)) return NVFP4_ERR_NULL;
  if (T > 0 && (!topk_ids || !row_to_tk || !tk_to_row || !x != !rows)) return NVFP4_ERR_NULL;
  if (!aligned16(x) || !aligned16(rows) || !aligned16(workspace) || !aligned_to(topk_ids, 4) ||
      !aligned_to(expert_offsets, 4) || !aligned_to(row_to_tk, 4) || !aligned_to(tk_to_row, 4) || !aligned_to(dev_err, 4))
    return NVFP4_ERR_ALIGN;
  if (x && x == rows) return NVFP4_ERR_ARG;
  if (workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  // a short list's workgroups all read the ids while others write the maps
  if (T > 0 && (row_to_tk == tk_to_row || expert_offsets == row_to_tk || expert_offsets == tk_to_row ||
                topk_ids == row_to_tk || topk_ids == tk_to_row || topk_ids == expert_offsets))
    return NVFP4_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n = T * (int64_t)k;
  const int words = (int)(H * (x_dtype == NVFP4_IN_F32 ? 4 : 2) / 16);
  const uint4* src = static_cast<const uint4*>(x);
  uint4* dst = static_cast<uint4*>(rows);
  if (n <= mp::kShort) {                          // T = 0: one workgroup, which writes the offsets
    const int per = (int)std::clamp<int64_t>((T + 255) / 256, 1, mp::kShortTokens);
    mp::permute_short_kernel<<<(unsigned)std::max<int64_t>(1, (T + per - 1) / per), kRouteThreads, 0, s>>>(
        src, (int)T, words, topk_ids, k, E, per, dst, expert_offsets, row_to_tk, tk_to_row, dev_err);
    return launch_status();
  }
  const int chunks = plan_chunks(n, mp::kChunkLog);
  int32_t* table = static_cast<int32_t*>(workspace);        // [chunks][E]
  int32_t* total = table + (int64_t)chunks * E;             // [E]
  int32_t* rank = total + E;                                // [n]
  route_rank_kernel<<<chunks, kPlanThreads, 0, s>>>(topk_ids, (int)n, E, mp::kChunkLog, table, rank, dev_err);
  const int rounds = mp::rounds_of(T, k);
  int group = 1;                                  // lanes that hold a short row, repeated over the wavefront
  while (group < kWave && group < words) group *= 2;
  const unsigned grid = (unsigned)((T + kRouteTokens * rounds - 1) / (kRouteTokens * rounds));
  if ((int64_t)chunks * E <= kCountTable) {
    mp::permute_kernel<true><<<grid, kRouteThreads, 0, s>>>(src, T, words, topk_ids, k, E, table, rank, nullptr, chunks,
        mp::kChunkLog, rounds, group, dst, expert_offsets, row_to_tk, tk_to_row);
  } else {
    mp::route_columns_kernel<<<(E + kWave - 1) / kWave, mp::kColumnWaves * 64, 0, s>>>(table, chunks, E, total);
    mp::permute_kernel<false><<<grid, kRouteThreads, 0, s>>>(src, T, words, topk_ids, k, E, table, rank, total, chunks,
        mp::kChunkLog, rounds, group, dst, expert_offsets, row_to_tk, tk_to_row);
  }
  return launch_status();
}

NVFP4MOE_API int moe_combine(const void* d, int32_t d_dtype, int64_t T, int32_t k, int64_t H, const int32_t* tk_to_row,
                             const float* topk_w, void* y, int32_t y_dtype, void* stream) {
  if (!mp::type_ok(d_dtype) || !mp::type_ok(y_dtype)) return NVFP4_ERR_ARG;
  if (const int bad = mp::check(T, k, H)) return bad;
  if (T * ((H + 511) / 512) > MOE_MAX_ROWS) return NVFP4_ERR_SHAPE;
  if (T == 0) return NVFP4_OK;
  if (!d || !tk_to_row || !y) return NVFP4_ERR_NULL;
  if (!aligned16(d) || !aligned16(y) || !aligned_to(tk_to_row, 4) || !aligned_to(topk_w, 4)) return NVFP4_ERR_ALIGN;
  if (d == y) return NVFP4_ERR_ARG;
  // at most 2^32 - 1024 lanes, by the limit above
  const unsigned grid = (unsigned)((T * (H / 8) + mp::kThreads - 1) / mp::kThreads);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool df = d_dtype == NVFP4_IN_F32, yf = y_dtype == NVFP4_IN_F32;
#define MP_COMBINE(D, Y) mp::combine_kernel<D, Y><<<grid, mp::kThreads, 0, s>>>(d, (int)T, k, (int)H, tk_to_row, topk_w, y)
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
  if (!aligned16(dy) || !aligned16(d) || !aligned16(dd) || !aligned_to(tk_to_row, 4) || !aligned_to(topk_w, 4) ||
      !aligned_to(dtopk_w, 4))
    return NVFP4_ERR_ALIGN;
  if (dd && (dd == d || dd == dy)) return NVFP4_ERR_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t R = T * (int64_t)k;
  const int lg = mp::log_lanes_for(H / 8), per = mp::kThreads >> lg;
  const unsigned grid = (unsigned)((R + per - 1) / per);
  const bool yf = dy_dtype == NVFP4_IN_F32, df = d_dtype == NVFP4_IN_F32;
  const int64_t bytes = T * H * (yf ? 4 : 2) + R * H * (df ? 4 : 2) * ((dtopk_w ? 1 : 0) + (dd ? 1 : 0));
  const bool streamed = bytes >= kLastLevelCache;
#define MP_BACKWARD(Y, D, S, A)                                                                                  \
  mp::combine_backward_kernel<Y, D, S, A><<<grid, mp::kThreads, 0, s>>>(dy, d, (int)R, k, (int)H, lg, tk_to_row, \
                                                                        topk_w, dd, dtopk_w)
#define MP_BACKWARD_BY(Y, D)                                                                            \
  do {                                                                                                  \
    if (H <= 8 << lg) streamed ? MP_BACKWARD(Y, D, true, 1) : MP_BACKWARD(Y, D, false, 1);              \
    else streamed ? MP_BACKWARD(Y, D, true, mp::kAhead) : MP_BACKWARD(Y, D, false, mp::kAhead);         \
  } while (0)
  if (yf) { if (df) MP_BACKWARD_BY(true, true); else MP_BACKWARD_BY(true, false); }
  else { if (df) MP_BACKWARD_BY(false, true); else MP_BACKWARD_BY(false, false); }
#undef MP_BACKWARD_BY
#undef MP_BACKWARD
  return launch_status();
}

}  // extern "C"
