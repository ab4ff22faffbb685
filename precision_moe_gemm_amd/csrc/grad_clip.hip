// The norm of the gradients over many tensors, and clipping by it, for gfx950.  Both stream the tensors
// once; clipping streams them a second time, in and out.  Bound by memory: 2.06 GB of a layer's gradients are
// clipped in 1.02 ms, 6.17 GB read and written at 6.05 TB/s.
//
// The tensors' addresses go to the kernels by value, kTensors a launch, so that no table has to be copied
// to the device first.  A launch's work is cut into pieces of kPiece bytes (131072: 1.06 ms).  For the norm,
// workgroup b of at most kPartials a launch (256: 1.18 ms, 2048: 1.04 ms) takes pieces b, b + grid, ... and adds
// its sum of squares to the one that workgroup b of the launches before it left: launches run one after another,
// so each has to fill the device by itself (2.15 GB as 6 tensors 333 us, as 400, 1000 and 4000 344, 377 and 550;
// with 1024 workgroups shared out over the launches 613, 1256 and 5160).  The clipping workgroups take one piece each (2048 workgroups that take many: 1.11
// ms for 1.09) and add the partial sums up themselves, all in the same order.  Loads run kAhead words ahead
// (1 instead of 4: 1.17 ms for 1.14).
//
// Where the tensors do not fit the 256 MB last-level cache, loads and stores are non-temporal (1.02 ms for
// 1.09).  Where they do, the second pass and the optimizer's read find them cached and ordinary ones are
// faster: with that read 117 us for 125 at 100 MB, 190 for 197 at 180 MB, 277 for 269 at 256 MB, 474 for 424
// at 400 MB.
//
// Squares of bf16 and float32 values are exact in float64, and their float64 sums, in an order that depends on
// the sizes and the alignment alone, are off by far less than a float32 step, so the norm is rounded once.
#include <algorithm>
#include <new>

#include "common.h"
#include "rows.h"

namespace nvfp4moe {
namespace gc {

constexpr int kTensors = 96;          // tensors a launch (the kernel arguments hold 4 KB)
constexpr int kThreads = 256;
constexpr int kPiece = 65536;         // bytes of a piece, 16-byte words of one tensor
constexpr int kPieceWords = kPiece / 16;
constexpr int kPartials = 1024;       // most norm workgroups of a launch, and partial sums of all of them
constexpr int kAhead = 4;

struct Table {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t numel[kTensors];
  int32_t first[kTensors + 1];        // the first piece of each tensor
  uint8_t f32[kTensors];
  int32_t n;
};

// Elements before the first 16-byte boundary of p.
__host__ __device__ inline int64_t head_of(const void* p, int64_t numel, int size) {
  const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / size;
  return h < numel ? h : numel;
}

// A piece: the 16-byte words [w0, w1) of a tensor behind its head; the first piece also has the head and
// the tail, elements that fill no word.
struct Piece {
  int j;
  int64_t head, words, w0, w1;
  bool first;
};

__device__ __forceinline__ Piece piece_of(const Table& t, int p) {
  int lo = 0, hi = t.n;               // the last tensor whose first piece is at or before p
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= p) lo = mid; else hi = mid;
  }
  Piece q;
  q.j = lo;
  const int size = t.f32[lo] ? 4 : 2;
  q.head = head_of(t.in[lo], t.numel[lo], size);
  q.words = (t.numel[lo] - q.head) * size / 16;
  q.w0 = (int64_t)(p - t.first[lo]) * kPieceWords;
  q.w1 = min(q.words, q.w0 + kPieceWords);
  q.first = p == t.first[lo];
  return q;
}

template <bool F32>
__device__ __forceinline__ double squares(uint4 v, double acc) {
  if constexpr (F32) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { const double d = __uint_as_float(w[j]); acc = __builtin_fma(d, d, acc); }
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double a = bf16_lo(w[j]), b = bf16_hi(w[j]);
      acc = __builtin_fma(a, a, acc);
      acc = __builtin_fma(b, b, acc);
    }
  }
  return acc;
}

template <bool F32, bool STREAM, int N>
__device__ __forceinline__ double piece_squares(const void* p, int64_t numel, const Piece& q) {
  constexpr int V = F32 ? 4 : 8;
  const uint4* words = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + q.head * (F32 ? 4 : 2));
  double acc = 0.0, part[kAhead] = {};
  int64_t w = q.w0 + threadIdx.x;
  for (; w + (kAhead - 1) * N < q.w1; w += kAhead * N) {
    uint4 r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) r[u] = load16<STREAM>(words + w + u * N);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) part[u] = squares<F32>(r[u], part[u]);
  }
  for (; w < q.w1; w += N) acc = squares<F32>(words[w], acc);
#pragma unroll
  for (int u = 0; u < kAhead; ++u) acc += part[u];
  if (q.first) {
    const int64_t tail = q.head + q.words * V, rest = q.head + numel - tail;   // head and tail elements
    for (int64_t i = threadIdx.x; i < rest; i += N) {
      const double d = load_one<F32>(p, i < q.head ? i : tail + (i - q.head));
      acc = __builtin_fma(d, d, acc);
    }
  }
  return acc;
}

// the workgroup's sum in thread 0
__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (unsigned w = 0; w < blockDim.x / kWave; ++w) s += lds[w];
  return s;
}

// used: the partial sums that launches before this one have written; the others are written here for the first time
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void squares_kernel(const Table t, int used, double* __restrict__ partial) {
  __shared__ double lds[kThreads / kWave];
  double acc = 0.0;
  for (int p = blockIdx.x; p < t.first[t.n]; p += gridDim.x) {
    const Piece q = piece_of(t, p);
    acc += t.f32[q.j] ? piece_squares<true, STREAM, kThreads>(t.in[q.j], t.numel[q.j], q)
                      : piece_squares<false, STREAM, kThreads>(t.in[q.j], t.numel[q.j], q);
  }
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = (int)blockIdx.x < used ? partial[blockIdx.x] + acc : acc;
}

// The norm from n partial sums, in every thread, in an order that is the same in every workgroup.
__device__ __forceinline__ double norm_of(const double* __restrict__ partial, int n, double* lds) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += partial[i];
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) lds[0] = __builtin_sqrt(acc);
  __syncthreads();
  return lds[0];
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const double* __restrict__ partial, int n, float* __restrict__ norm) {
  __shared__ double lds[kThreads / kWave];
  const double v = norm_of(partial, n, lds);
  if (threadIdx.x == 0) *norm = (float)v;
}

// x * c in float64, so that a factor below float32's normal range (a norm above 2^126) costs no bits
__device__ __forceinline__ float times(float x, double c) { return (float)((double)x * c); }

// out = in * c for one piece; words when in and out lie alike towards a 16-byte boundary, else element by element
// (10^8 float32 and 10^8 bf16 elements: 334 us and 453, the norm included)
template <bool F32, bool STREAM, int N>
__device__ __forceinline__ void scale_piece(const void* in, void* out, int64_t numel, const Piece& q, double c) {
  constexpr int V = F32 ? 4 : 8, size = F32 ? 4 : 2;
  const int64_t tail = q.head + q.words * V;
  if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(in) + q.head * size);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(out) + q.head * size);
    for (int64_t w0 = q.w0 + threadIdx.x; w0 < q.w1; w0 += kAhead * N) {
      uint4 r[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) r[u] = load16<STREAM>(src + min(w0 + u * N, q.w1 - 1));
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (w0 + u * N >= q.w1) continue;
        uint32_t x[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (F32) x[j] = __float_as_uint(times(__uint_as_float(x[j]), c));
          else x[j] = bf16x2_rne(times(bf16_lo(x[j]), c), times(bf16_hi(x[j]), c));
        }
        store16<STREAM>(dst + w0 + u * N, make_uint4(x[0], x[1], x[2], x[3]));
      }
    }
  } else {
    for (int64_t i = q.head + q.w0 * V + threadIdx.x; i < q.head + q.w1 * V; i += N)
      store_one<F32>(out, i, times(load_one<F32>(in, i), c));
  }
  if (q.first) {
    const int64_t rest = q.head + numel - tail;
    for (int64_t i = threadIdx.x; i < rest; i += N) {
      const int64_t at = i < q.head ? i : tail + (i - q.head);
      store_one<F32>(out, at, times(load_one<F32>(in, at), c));
    }
  }
}

// min(1, max_norm / (norm + 1e-6)), NaN for a NaN norm; max_norm = inf asks for the norm alone: 1, also where the
// norm is inf (inf / inf would be NaN) or NaN
__device__ __forceinline__ double factor_of(double norm, double max_norm) {
  if (max_norm == INFINITY) return 1.0;
  const double ratio = max_norm / (norm + 1e-6);
  return ratio >= 1.0 ? 1.0 : ratio;
}

template <bool STREAM, int N>
__device__ __forceinline__ void scale_piece_of(const Table& t, const Piece& q, double c) {
  if (c == 1.0 && t.in[q.j] == t.out[q.j]) return;    // clipped in place by a factor of 1: as it is
  if (t.f32[q.j]) scale_piece<true, STREAM, N>(t.in[q.j], t.out[q.j], t.numel[q.j], q, c);
  else scale_piece<false, STREAM, N>(t.in[q.j], t.out[q.j], t.numel[q.j], q, c);
}

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void scale_kernel(const Table t, const double* __restrict__ partial, int n,
                                                         double max_norm, float* __restrict__ norm) {
  __shared__ double lds[kThreads / kWave];
  const double v = norm_of(partial, n, lds);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  scale_piece_of<STREAM, kThreads>(t, piece_of(t, blockIdx.x), factor_of(v, max_norm));
}

// At most two pieces (a tensor of up to 128 KB, or two of up to 64): one workgroup takes the norm and clips, in one
// launch.  One tensor of 8 KB 4.7 us for 5.8, of 128 KB 9.0 for 8.3, and 8.5 and 8.8 for 11.5 and 11.3 with the
// host's part; a third piece and every further one would take it 2 us more, eight tensors 18 for 7.
constexpr int kSmallThreads = 1024;
constexpr int kSmallPieces = 2;
template <bool CLIP>
__global__ __launch_bounds__(kSmallThreads) void small_kernel(const Table t, double max_norm, float* __restrict__ norm) {
  __shared__ double lds[kSmallThreads / kWave];
  const int pieces = t.first[t.n];
  double acc = 0.0;
  for (int p = 0; p < pieces; ++p) {
    const Piece q = piece_of(t, p);
    acc += t.f32[q.j] ? piece_squares<true, false, kSmallThreads>(t.in[q.j], t.numel[q.j], q)
                      : piece_squares<false, false, kSmallThreads>(t.in[q.j], t.numel[q.j], q);
  }
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    lds[0] = __builtin_sqrt(acc);
    *norm = (float)lds[0];
  }
  __syncthreads();
  if constexpr (CLIP) {
    const double c = factor_of(lds[0], max_norm);
    for (int p = 0; p < pieces; ++p) scale_piece_of<false, kSmallThreads>(t, piece_of(t, p), c);
  }
}

// ------------------------------------------------------------------ host
int check(const void* const* in, const int32_t* dtype, const int64_t* numel, int32_t n) {
  if (n < 0 || n > MOE_MAX_TENSORS) return NVFP4_ERR_SHAPE;
  if (n && (!in || !dtype || !numel)) return NVFP4_ERR_NULL;
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) {
    if (dtype[i] != NVFP4_IN_BF16 && dtype[i] != NVFP4_IN_F32) return NVFP4_ERR_ARG;
    if (numel[i] < 0 || numel[i] > MOE_MAX_GRAD_BYTES) return NVFP4_ERR_SHAPE;
    bytes += numel[i] * (dtype[i] == NVFP4_IN_F32 ? 4 : 2);
    if (bytes > MOE_MAX_GRAD_BYTES) return NVFP4_ERR_SHAPE;
    if (numel[i] && !in[i]) return NVFP4_ERR_NULL;
    if (!aligned_to(in[i], dtype[i] == NVFP4_IN_F32 ? 4 : 2)) return NVFP4_ERR_ALIGN;
  }
  return NVFP4_OK;
}

// Whether an output overlaps another output, or an input other than its own tensor's.
int overlaps(const void* const* in, void* const* out, const int32_t* dtype, const int64_t* numel, int32_t n) {
  struct Range { uintptr_t lo, hi; bool out; };
  Range* r = new (std::nothrow) Range[2 * (size_t)n + 1];
  if (!r) return NVFP4_ERR_SHAPE;
  size_t m = 0;
  for (int i = 0; i < n; ++i) {
    const uintptr_t bytes = (uintptr_t)numel[i] * (dtype[i] == NVFP4_IN_F32 ? 4 : 2);
    if (!bytes) continue;
    const uintptr_t o = reinterpret_cast<uintptr_t>(out[i]), a = reinterpret_cast<uintptr_t>(in[i]);
    r[m++] = {o, o + bytes, true};
    if (o != a) r[m++] = {a, a + bytes, false};
  }
  std::sort(r, r + m, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;
  int bad = NVFP4_OK;
  for (size_t i = 0; i < m; ++i) {
    if (r[i].lo < (r[i].out ? any : outs)) bad = NVFP4_ERR_ARG;
    any = std::max(any, r[i].hi);
    if (r[i].out) outs = std::max(outs, r[i].hi);
  }
  delete[] r;
  return bad;
}

// Tensors [i0, n) into a table until it is full; returns the first that is not in it.  Empty tensors are left
// out.  (MOE_MAX_GRAD_BYTES and MOE_MAX_TENSORS make fewer than 2^24 pieces, as many workgroups of 256 threads
// as a launch holds.)
int fill(Table& t, const void* const* in, void* const* out, const int32_t* dtype, const int64_t* numel, int i0, int n) {
  t.n = 0;
  t.first[0] = 0;
  int i = i0;
  for (; i < n && t.n < kTensors; ++i) {
    if (!numel[i]) continue;
    const int j = t.n, size = dtype[i] == NVFP4_IN_F32 ? 4 : 2;
    const int64_t words = (numel[i] - head_of(in[i], numel[i], size)) * size / 16;
    const int64_t pieces = std::max<int64_t>(1, (words + kPieceWords - 1) / kPieceWords);
    t.in[j] = in[i];
    t.out[j] = out ? out[i] : nullptr;
    t.numel[j] = numel[i];
    t.f32[j] = dtype[i] == NVFP4_IN_F32;
    t.first[j + 1] = t.first[j] + (int)pieces;
    t.n = j + 1;
  }
  return i;
}

int run(const void* const* in, void* const* out, const int32_t* dtype, const int64_t* numel, int32_t n, double max_norm,
        float* norm, double* partial, hipStream_t s) {
  Table t;
  int used = 0;
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) bytes += numel[i] * (dtype[i] == NVFP4_IN_F32 ? 4 : 2);
  if (fill(t, in, out, dtype, numel, 0, n) == n && t.n && t.first[t.n] <= kSmallPieces) {
    if (out) small_kernel<true><<<1, kSmallThreads, 0, s>>>(t, max_norm, norm);
    else small_kernel<false><<<1, kSmallThreads, 0, s>>>(t, max_norm, norm);
    return launch_status();
  }
  const bool stream = bytes >= kLastLevelCache;
  for (int i = 0; i < n;) {
    i = fill(t, in, out, dtype, numel, i, n);
    if (!t.n) break;
    const int grid = std::min(kPartials, t.first[t.n]);
    if (stream) squares_kernel<true><<<grid, kThreads, 0, s>>>(t, used, partial);
    else squares_kernel<false><<<grid, kThreads, 0, s>>>(t, used, partial);
    used = std::max(used, grid);
  }
  if (!out || !used) {
    norm_kernel<<<1, kThreads, 0, s>>>(partial, used, norm);
    return launch_status();
  }
  for (int i = 0; i < n;) {
    const bool first = i == 0;
    i = fill(t, in, out, dtype, numel, i, n);
    if (!t.n) break;
    float* to = first ? norm : nullptr;
    if (stream) scale_kernel<true><<<t.first[t.n], kThreads, 0, s>>>(t, partial, used, max_norm, to);
    else scale_kernel<false><<<t.first[t.n], kThreads, 0, s>>>(t, partial, used, max_norm, to);
  }
  return launch_status();
}

}  // namespace gc
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" {

NVFP4MOE_API size_t moe_grad_workspace_size(int32_t n) {
  if (n < 0 || n > MOE_MAX_TENSORS) return 0;
  return gc::kPartials * sizeof(double);
}

NVFP4MOE_API int moe_grad_norm(const void* const* grads, const int32_t* dtypes, const int64_t* numel, int32_t n,
                               float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int bad = gc::check(grads, dtypes, numel, n)) return bad;
  if (!norm || !workspace) return NVFP4_ERR_NULL;
  if (!aligned16(workspace) || !aligned_to(norm, 4)) return NVFP4_ERR_ALIGN;
  if (workspace_bytes < moe_grad_workspace_size(n)) return NVFP4_ERR_WORKSPACE;
  return gc::run(grads, nullptr, dtypes, numel, n, 0.0, norm, static_cast<double*>(workspace),
                 static_cast<hipStream_t>(stream));
}

NVFP4MOE_API int moe_grad_clip(const void* const* grads, void* const* out, const int32_t* dtypes, const int64_t* numel,
                               int32_t n, double max_norm, float* norm, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (!(max_norm >= 0.0)) return NVFP4_ERR_ARG;
  if (const int bad = gc::check(grads, dtypes, numel, n)) return bad;
  if (!norm || !workspace || (n && !out)) return NVFP4_ERR_NULL;
  if (const int bad = gc::check(out, dtypes, numel, n)) return bad;
  if (!aligned16(workspace) || !aligned_to(norm, 4)) return NVFP4_ERR_ALIGN;
  if (workspace_bytes < moe_grad_workspace_size(n)) return NVFP4_ERR_WORKSPACE;
  if (const int bad = gc::overlaps(grads, out, dtypes, numel, n)) return bad;
  return gc::run(grads, out, dtypes, numel, n, max_norm, norm, static_cast<double*>(workspace),
                 static_cast<hipStream_t>(stream));
}

}  // extern "C"
