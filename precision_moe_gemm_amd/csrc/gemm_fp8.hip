// FP8 (E4M3fn) grouped expert GEMM with one FP32 scale per 128 elements of an
// activation row and per 128 x 128 block of a weight, gfx950:
//     c[r][n] = sum_j sa[j][r] * sw[e][n / 128][j] * sum_{k in block j} a[r][k] w[e][n][k].
// A block's inner sum starts from zero on the matrix cores; its result is scaled
// by sa * sw and added to the FP32 accumulator by FMAs on the vector unit, which
// run under the next blocks' matrix instructions.
//
// Which matrix instruction forms the block's sum goes by the output's type.  The
// FP8 one (v_mfma_f32_16x16x128_f8f6f4, twice the FP16 rate) aligns the products
// of each 8 consecutive k to the largest of them and cuts them off 13 bits below
// its leading bit before they reach the FP32 sum (measured: products of the same
// aligned 8 keep 2^-13 of the largest, others 2^-23; truncation, not rounding).
// On Gaussian data that is 1.4e-5 of the result's 2-norm, with outliers 6e-5:
// far below half a BF16 step (2^-9 to 2^-8), too much for an FP32 result.  So BF16
// outputs take the FP8 instruction; FP32 outputs take FP16 ones on codes converted
// in registers (E4M3 fits FP16 exactly; 8e-9 on the same data).
//
// Two kernels.  Many rows per expert: tiles of up to 256 rows x 256 columns through
// LDS (grouped_gemm_kernel).  Few rows per expert: the weights are read once and
// are all that matters, straight into registers (rows_kernel).  Both form the same
// products in the same order, so a row's bits depend neither on the kernel nor on
// how many rows its expert has.
//
// Measured.  Tiles, BF16 out: 128 experts of 1536 x 2048 over 32768 gathered rows 187 us
// (1100 TFLOP/s; 512 MB at 2.7 TB/s), one of 5120 x 2048 over 4096 rows 69 us (1240),
// 8192^3 572 us (1920).  Of the grouped product's time the loads into LDS are the longer part
// (165 us with the matrix instructions left out, 137 with the loads left out): 1.2 GB or 29
// GB/s a CU.  A K-step's loads, some 50 KB here, where a tile holds about 136 rows, are requested
// a step ahead and waited for in full, so no more than one step's are ever in flight.
// FP32 out: 109 us (785 TFLOP/s) for the 5120 x 2048 product, whose 440 tiles fill the second of
// two rounds to 72 %, 1125 us (980) for 8192^3: a SIMD's two wavefronts convert, multiply and add
// at nearly the same time, so matrix and vector cycles (1.05 and 0.9 million of 2.3) mostly add up;
// without the conversions it takes 7 % less, with a quarter of the FMAs 4 %.
// The FP8 tile kernel fills its 256 registers and spills 2, the form for N not a multiple of 8
// 21 (with 6 for the 2, gate_up took 241 us for 189).
// Rows: one token through 8 of 128 experts of 1536 x 2048, 25 MB, 9.6 us (5 at the copy's rate; a
// launch, then offsets, map entries, and rows and weights, each behind the one before); 128 rows
// over all 128 of them, 403 MB, 48 us, the weights partly from the last-level cache; 488 rows over
// 128 experts of 2048 x 768, FP32 out, 42 us (4.8 TB/s).
#include "fp8.h"
#include "lds_dma.h"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace nvfp4moe {
namespace g8 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));

constexpr int BK = kFp8Block;

// An operand's fragment over one block of 128: lane (l16 = lane % 16, g = lane / 16)
// holds 32 bytes of row l16, as read (FP8) or converted to FP16.  Which 32 of the
// 128 is free as long as both operands take the same; these kernels take the
// 16-byte chunks g and g + 4.
template <bool F16>
struct Frag {
  v8i v;
  __device__ __forceinline__ explicit Frag(v8i raw) : v(raw) {}
};
template <>
struct Frag<true> {
  halfx8 v[4];
  __device__ __forceinline__ explicit Frag(v8i raw) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const halfx2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[2 * s], 1.0f, false);
      const halfx2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[2 * s], 1.0f, true);
      const halfx2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[2 * s + 1], 1.0f, false);
      const halfx2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw[2 * s + 1], 1.0f, true);
      v[s] = halfx8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
  }
};

// D[n][m] = sum over the block of W[n][k] A[m][k]; the lane receives rows n =
// 4g .. 4g+3 of column m = l16.
__device__ __forceinline__ floatx4 block_sum(const Frag<false>& w, const Frag<false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ floatx4 block_sum(const Frag<true>& w, const Frag<true>& a) {
  floatx4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[s], a.v[s], p, 0, 0, 0);
  return p;
}

__device__ __forceinline__ v8i join(v4i a, v4i b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A block's term is sa sw p, p its sum of code products (2^-18 <= |p| < 2^25, or 0), added as
// fma(p, fl(sa sw), acc).  Where fl(sa sw) leaves the normal range it has lost bits or is zero or
// infinite, while the term may be an ordinary number: then the mantissas are multiplied and the
// exponents added, and the term is rounded once more only if it is itself below that range.
struct Scale {
  float s, m;
  int e;
  bool far;
  __device__ __forceinline__ Scale(float sa, float sw)
      : s(sa * sw), m(__builtin_amdgcn_frexp_mantf(sa) * __builtin_amdgcn_frexp_mantf(sw)),
        e(__builtin_amdgcn_frexp_expf(sa) + __builtin_amdgcn_frexp_expf(sw)),
        far(__builtin_amdgcn_classf(s, 0x2F4) && sa != 0.0f && sw != 0.0f) {}   // subnormal, zero or infinite
  __device__ __forceinline__ float add(float p, float acc) const {
    return far ? acc + __builtin_ldexpf(p * m, e) : __builtin_fmaf(p, s, acc);
  }
};
// The sum of the two exponents, as an unsigned distance from the least one whose products are
// all normal numbers: some product may be out of range if it is above kNear.
constexpr uint32_t kNear = 251;
__device__ __forceinline__ uint32_t exponents(float sa, float sw) {
  return (uint32_t)(__builtin_amdgcn_frexp_expf(sa) + __builtin_amdgcn_frexp_expf(sw) + 124);
}

// The sums of 16 columns x 16 rows, from memory, each term in the form its scales call for: lane
// (l16, g) gives column l16's weights and row l16's activations, and receives columns 4g .. 4g+3
// of row l16.  Both kernels go back to it for rows that have met a scale product out of range
// (never in practice, so it is short rather than fast).
template <bool F16>
__device__ __forceinline__ floatx4 far_sums(const uint8_t* arow, const float* sa, int a_rows, const uint8_t* wrow,
                                            const float* sw, int nk, int K, int g) {
  floatx4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int kb = 0; kb < nk; ++kb) {
    const int k = kb * BK + 16 * g;
    auto load = [&](const uint8_t* row) __attribute__((always_inline)) -> v8i {   // chunks past K are zero
      const v4i z = {0, 0, 0, 0};
      return join(k < K ? *reinterpret_cast<const v4i*>(row + k) : z,
                  k + 64 < K ? *reinterpret_cast<const v4i*>(row + k + 64) : z);
    };
    const Scale s(sa[(int64_t)kb * a_rows], sw[kb]);
    const floatx4 p = block_sum(Frag<F16>(load(wrow)), Frag<F16>(load(arow)));
#pragma unroll
    for (int v = 0; v < 4; ++v) r[v] = s.add(p[v], r[v]);
  }
  return r;
}

// expert offsets clamped into [0, Rc]: malformed offsets give wrong rows but no
// access outside the buffers
__device__ __forceinline__ int off_at(const int32_t* __restrict__ offsets, int Rc, int e) {
  return min(max(offsets[e], 0), Rc);
}

// ------------------------------------------------------------------ many rows per expert
// A workgroup of 8 wavefronts (2 x 4) computes up to BM x 256, a wavefront up to
// 16 FM x 64 of it.  BM is 256 for the FP8 kernel and 192 for the FP16 one, whose
// fragments take twice the registers.
constexpr int BN = 256;
constexpr int kTileCost = 96;                  // rows' worth of a tile's cost that does not scale with its rows:
                                               // at 16 / 96 / 256 gate_up takes 313 / 189 / 199 us, the QKV product
                                               // 108 / 70 / 70 (BF16 out), down 234 / 177 / 173, a Zipf gate_up 325 / 206 / 203
constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int FN = 4, WN = 64;
constexpr int kWI = BN / 8 / kWaves;           // weight load instructions per wavefront and K-step (8 rows each)
constexpr int kWSlots = 2, kASlots = 2;        // K-steps in LDS
constexpr uint32_t kOutOfRange = 0x80000000u;  // buffer offset that the range check drops

// Tile heights to choose from: BM and the smaller multiples of 64.  Against BM alone, in
// BF16: 187 us for 193 to 204 (grouped), 67 for 75 (5120 x 2048 over 4096 rows), measured
// before the check of the scale products.
constexpr int kNumHeights = 5;
__host__ __device__ constexpr int height(int bm, int i) { return i == 0 ? bm : 64 * ((bm - 1) / 64 + 1 - i) > 64 ? 64 * ((bm - 1) / 64 + 1 - i) : 64; }

template <int FM>
struct __align__(16) Smem {
  static constexpr int BM = 32 * FM, kSaWaves = (BM + 63) / 64, kSa = 64 * kSaWaves;
  uint8_t a[kASlots][BM * BK];
  uint8_t w[kWSlots][BN * BK];
  float sa[kASlots][kSa];
  float sw[kASlots][64];      // two weight blocks' scales
  int32_t map[2][kSa];        // gathered operand: the routing map of a tile's rows
  int tile_start[NVFP4MOE_MAX_EXPERTS + 1];   // first m-tile of each expert
  int off[NVFP4MOE_MAX_EXPERTS + 1];          // its first row
  int64_t cost[kNumHeights];
  int far[kWaves];            // the wavefront met a scale product that may be out of range
};
static_assert(sizeof(Smem<10>) <= 160 * 1024, "LDS");

// Waits until at most n of this wavefront's loads and stores are outstanding (or
// fewer: n is rounded down to one of the counts below).
__device__ __forceinline__ void wait_vmcnt(int n) {
#define G8_W(v) __builtin_amdgcn_s_waitcnt(0x0F70 | ((v) & 15) | ((v) >> 4 << 14))
  if (n >= 16) G8_W(16);
  else if (n >= 8) G8_W(8);
  else if (n >= 4) G8_W(4);
  else G8_W(0);
#undef G8_W
}

struct Tile {
  int e, m0, rows, n0;
};

// Tile L; `from` is an expert at or before the tile's.  An expert's tiles run in
// groups of kGroupM m-tiles, column by column: the 32 workgroups of an XCD, on
// consecutive tiles, then share both operands' slabs in its L2 (8192^3: 556 us in groups
// of 4, 575 of 1, 560 of 8).
constexpr int kGroupM = 4;
__device__ __forceinline__ Tile tile_at(int L, int from, int n_tiles, const int* tile_start, const int* offs, int E) {
  const int tm = L / n_tiles, lane = lane_id();
  // the last expert that starts at or before m-tile tm, 64 experts at a look
  Tile t;
  t.e = from;
  for (;;) {
    const int x = t.e + 1 + lane;
    const int n = __popcll(__ballot(x < E && tile_start[min(x, E)] <= tm));
    t.e += n;
    if (n < kWave) break;
  }
  const int o0 = __builtin_amdgcn_readfirstlane(offs[t.e]), o1 = __builtin_amdgcn_readfirstlane(offs[t.e + 1]);
  const int s0 = __builtin_amdgcn_readfirstlane(tile_start[t.e]);
  const int nt = __builtin_amdgcn_readfirstlane(tile_start[t.e + 1]) - s0;
  const int idx = L - s0 * n_tiles, b = idx / (kGroupM * n_tiles), r = idx - b * kGroupM * n_tiles;
  const int h = min(kGroupM, nt - b * kGroupM), tn = r / h;
  // the expert's rows split evenly over its m-tiles, in 16-row groups (no tile
  // is empty, none taller than the launch's height)
  const int per = ((o1 - o0 + nt - 1) / nt + 15) & ~15;
  t.m0 = o0 + (b * kGroupM + r - tn * h) * per;
  t.rows = max(0, min(per, o1 - t.m0));
  t.n0 = tn * BN;
  return t;
}

// The wavefront's part of its tiles once more, in the 16-row groups that have a scale product out
// of range.  A function of its own: inlined, its live values make the tile loop spill (gate_up 241
// us for 189).
template <bool BF16OUT, int FM>
__device__ __attribute__((noinline)) void far_tiles(const Smem<FM>& sm, int begin, int end, int step, const uint8_t* a,
                                                    const float* sa, int a_rows, const int32_t* a_map, int a_div, int E,
                                                    const uint8_t* w, const float* sw, int N, int K, void* c) {
  const int lane = lane_id(), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int nk = (K + BK - 1) / BK, nnb = (N + BK - 1) / BK;
  Tile t{0, 0, 0, 0};
  for (int L = begin; L < end; L += step) {
    t = tile_at(L, t.e, (N + BN - 1) / BN, sm.tile_start, sm.off, E);
    const int nb = (t.n0 + WN * wn) / BK;
    if (nb >= nnb) continue;
    const float* psw = sw + ((int64_t)t.e * nnb + nb) * nk;
    for (int r0 = 16 * wm; r0 < t.rows; r0 += 32) {
      const int m = t.m0 + min(r0 + l16, t.rows - 1);
      const int64_t src = a_map ? min(max(a_map[m], 0) / a_div, a_rows - 1) : m;
      uint32_t reach = 0;
      for (int kb = g; kb < nk; kb += 4) reach = max(reach, exponents(sa[(int64_t)kb * a_rows + src], psw[kb]));
      if (__builtin_amdgcn_ballot_w64(reach > kNear) == 0) continue;
      for (int n = t.n0 + WN * wn; n < min(N, t.n0 + WN * wn + WN); n += 16) {
        const int64_t col = (int64_t)t.e * N + min(n + l16, N - 1);
        const floatx4 r = far_sums<!BF16OUT>(a + src * K, sa + src, a_rows, w + col * K, psw, nk, K, g);
        if (r0 + l16 >= t.rows) continue;
        const int64_t at = (int64_t)m * N + n + 4 * g;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (n + 4 * g + v >= N) break;
          if constexpr (BF16OUT) static_cast<uint16_t*>(c)[at + v] = (uint16_t)bf16x2_rne(r[v], 0.0f);
          else static_cast<float*>(c)[at + v] = r[v];
        }
      }
    }
  }
}

// WHOLE: rows of c are whole 16-byte pieces
template <bool BF16OUT, bool WHOLE, int FM>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void grouped_gemm_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa, int a_rows,
                         const int32_t* __restrict__ a_map, int a_div,
                         const int32_t* __restrict__ offsets, int E, int Rc,
                         const uint8_t* __restrict__ w, const float* __restrict__ sw, int N, int K,
                         void* __restrict__ c) {
  constexpr bool F16 = !BF16OUT;
  constexpr int BM = 32 * FM, kSaWaves = Smem<FM>::kSaWaves;
  constexpr int kAI = (BM / 8 + kWaves - 1) / kWaves;   // activation load instructions per wavefront
  __shared__ Smem<FM> sm;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, g = lane >> 4;
  const int n_tiles = (N + BN - 1) / BN;

  for (int e = tid; e <= E; e += kThreads) sm.off[e] = off_at(offsets, Rc, e);
  if (tid < kWaves) sm.far[tid] = 0;
  __syncthreads();
  if (wave < kNumHeights) {
    // Tile height: the candidate with the smallest estimated critical path,
    // (tiles per workgroup) x (height + kTileCost); one wavefront each.
    const int h = height(BM, wave);
    int mt = 0;
    for (int e = lane; e < E; e += kWave) mt += max(0, sm.off[e + 1] - sm.off[e] + h - 1) / h;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) mt += __shfl_xor(mt, off, kWave);
    const int G = gridDim.x, xg = (G & 7) == 0 ? 8 : 1;
    const int64_t per = ((int64_t)mt * n_tiles + xg - 1) / xg, wgs = G / xg;
    if (lane == 0) sm.cost[wave] = (per + wgs - 1) / wgs * (h + kTileCost);
  }
  __syncthreads();
  if (wave == 0) {
    int best = BM;
    int64_t best_cost = sm.cost[0];
#pragma unroll
    for (int q = 1; q < kNumHeights; ++q)   // ties go to the taller
      if (sm.cost[q] < best_cost) {
        best_cost = sm.cost[q];
        best = height(BM, q);
      }
    int carry = 0;
    int64_t sum = 0;
    for (int e0 = 0; e0 < E; e0 += kWave) {
      const int e = e0 + lane;
      const int v = e < E ? max(0, sm.off[e + 1] - sm.off[e] + best - 1) / best : 0;
      int incl = v;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int y = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += y;
      }
      if (e < E) sm.tile_start[e] = carry + incl - v;
      const int here = __shfl(incl, kWave - 1, kWave);
      carry += here;
      sum += here;
    }
    // offsets that fall make more tiles than the rows can: no tile then, so that the
    // tile numbers stay within the range that the host checked
    if (lane == 0) sm.tile_start[E] = sum <= Rc / best + E ? carry : 0;
  }
  __syncthreads();

  const int total = __builtin_amdgcn_readfirstlane(sm.tile_start[E]) * n_tiles;
  int begin, end, step;
  if ((gridDim.x & 7) == 0) {
    const int per = (total + 7) / 8;
    const int xcd = blockIdx.x & 7;
    begin = xcd * per + (int)(blockIdx.x >> 3);
    end = min(total, (xcd + 1) * per);
    step = gridDim.x >> 3;
  } else {
    begin = blockIdx.x;
    end = total;
    step = gridDim.x;
  }
  if (begin >= end) return;
  const int nk = (K + BK - 1) / BK, tail = K & (BK - 1);
  const int nnb = (N + BK - 1) / BK;
  auto find = [&](int L, int from) __attribute__((always_inline)) {
    return tile_at(L, from, n_tiles, sm.tile_start, sm.off, E);
  };

  // ------------------------------------------------------------ loads
  // A load instruction q of an operand fills 1 KiB, rows 8q .. 8q+7: lane i gives
  // row 8q + i / 8, physical 16-byte chunk i % 8, which holds logical chunk
  // (i % 8) ^ (row / 2 mod 8) (see mma_step).  Wavefront v takes q = v, v + 8, ..;
  // its lanes' logical chunk is the same in all of them.
  const int chunk = 16 * ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7));
  // the last K-step's chunks past K read the row's first chunk of that step
  // instead (in bounds); the compute side clears them
  const uint32_t back = tail && chunk >= tail ? chunk : 0;
  const int row8 = 8 * wave + (lane >> 3);

  // Weights: the next K-step to load is step wk of tile wL, two steps ahead of
  // the one being computed (w_cols = 0: no tile left).  The cursor moves to the
  // next tile in next_w, outside the K-loop.
  int wL = begin - step, wk = 0, w_e = 0, w_cols = 0;
  const uint8_t* pw = w;
  uint32_t off_w[kWI];
  auto next_w = [&]() __attribute__((always_inline)) {
    wL += step;
    wk = 0;
    w_cols = 0;
    if (wL >= end) return;
    const Tile t = find(wL, w_e);
    w_e = t.e;
    w_cols = min(BN, N - t.n0);
#pragma unroll
    for (int u = 0; u < kWI; ++u) off_w[u] = (uint32_t)min(row8 + 64 * u, w_cols - 1) * (uint32_t)K + chunk;
    pw = w + ((int64_t)t.e * N + t.n0) * K;
  };
  auto issue_w = [&](int slot) __attribute__((always_inline)) -> int {   // returns the instructions issued
    const uint32_t dst = lds_addr(sm.w[0]) + slot * (BN * BK) + wave * 1024;
    const uint32_t bk = wk == nk - 1 ? back : 0;
    int n = 0;
#pragma unroll
    for (int u = 0; u < kWI; ++u)
      if (8 * wave + 64 * u < w_cols) {
        lds_dma16(pw, off_w[u] - bk, dst + u * kWaves * 1024);
        ++n;
      }
    pw += BK;
    ++wk;
    return n;
  };

  // Activations: step ak of tile at, one step ahead of the one being computed
  // (at.rows = 0: no tile left).  The first kSaWaves wavefronts also load the
  // scales of 64 rows each, the next one those of the tile's two weight column
  // blocks.  A gathered operand's map entries for the tile after it are on their
  // way into LDS meanwhile: row m of the tile reads row a_map[m] / a_div of a,
  // clamped into a (an invalid entry reads a wrong row, never outside).
  int aL = begin - step, ak = 0, abuf = 0;
  Tile at{0, 0, 0, 0}, an = find(begin, 0);
  const uint8_t* pa = a;
  const float* ps = sa;
  uint32_t off_a[kAI], off_s = 0;
  auto issue_map = [&](const Tile& t, int buf) __attribute__((always_inline)) {
    if (a_map && 64 * wave < t.rows)
      lds_dma4(a_map + t.m0, 4 * min(64 * wave + lane, t.rows - 1), lds_addr(sm.map[0]) + (buf * Smem<FM>::kSa + 64 * wave) * 4);
  };
  auto next_a = [&]() __attribute__((always_inline)) {
    aL += step;
    ak = 0;
    at.rows = 0;
    if (aL >= end) return;
    at = an;
    auto src = [&](int r) __attribute__((always_inline)) -> uint32_t {
      const int m = min(r, at.rows - 1);
      return a_map ? (uint32_t)min(max(sm.map[abuf][m], 0) / a_div, a_rows - 1) : (uint32_t)m;
    };
#pragma unroll
    for (int u = 0; u < kAI; ++u) off_a[u] = src(row8 + 64 * u) * (uint32_t)K + chunk;
    pa = a_map ? a : a + (int64_t)at.m0 * K;
    if (wave < kSaWaves) {
      ps = a_map ? sa : sa + at.m0;
      off_s = 4 * src(64 * wave + lane);
    } else {
      const int nb = at.n0 / BK;
      ps = sw + ((int64_t)at.e * nnb + nb) * nk;
      off_s = 4 * nk * min(min(lane, 1), nnb - 1 - nb);
    }
    abuf ^= 1;
    if (aL + step < end) {
      an = find(aL + step, at.e);
      issue_map(an, abuf);
    }
  };
  auto issue_a = [&](int slot) __attribute__((always_inline)) {
    const uint32_t dst = lds_addr(sm.a[0]) + slot * (BM * BK) + wave * 1024;
    const uint32_t bk = ak == nk - 1 ? back : 0;
#pragma unroll
    for (int u = 0; u < kAI; ++u)
      if (8 * wave + 64 * u < at.rows) lds_dma16(pa, off_a[u] - bk, dst + u * kWaves * 1024);
    if (wave < kSaWaves) {
      if (64 * wave < at.rows) lds_dma4(ps, off_s, lds_addr(sm.sa[0]) + (slot * Smem<FM>::kSa + 64 * wave) * 4);
    } else if (wave == kSaWaves && at.rows > 0) {
      lds_dma4(ps, off_s, lds_addr(sm.sw[0]) + slot * 256);
    }
    pa += BK;
    ps += wave < kSaWaves ? a_rows : 1;
    ++ak;
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // Fragments.  A read gives lane (l16, g) the chunks g and g + 4 of row l16 of
  // the fragment, each at its row's physical place, chunk ^ (row / 2 mod 8): a
  // 16-byte LDS read is served 16 lanes at a time, here 16 rows with chunk g from
  // one half and g ^ 1 from the other, and the XOR puts those on 16 different bank
  // groups.  In a tile's last K-step the chunks past K are cleared in registers.
  const int pc0 = 16 * (g ^ (l16 >> 1)), pc1 = 16 * ((g + 4) ^ (l16 >> 1));
  auto frag = [&](const uint8_t* row) __attribute__((always_inline)) -> v8i {
    return join(*reinterpret_cast<const v4i*>(row + pc0), *reinterpret_cast<const v4i*>(row + pc1));
  };
  auto clear_tail = [&](v8i& f) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < 8; ++x) f[x] = 16 * (g + (x & 4)) < tail ? f[x] : 0;
  };
  // One K-step.  Row fragments go FB at a time: a group past the wavefront's rows
  // is skipped, a partial one computed whole (the stage's other rows are whatever
  // it held, their results are never stored); the next group's reads are issued
  // before this one's matrix instructions.
  constexpr int FB = F16 ? 1 : 2;
  auto mma_step = [&](int slot, int nf, bool clear) __attribute__((always_inline)) {
    const uint8_t* wrow = sm.w[0] + slot * (BN * BK) + (WN * wn + l16) * BK;
    const uint8_t* arow = sm.a[0] + slot * (BM * BK) + (16 * wm + l16) * BK;
    const float* sav = sm.sa[0] + slot * Smem<FM>::kSa + 16 * wm + l16;
    v8i wr[FN], ar[FB];
    float sr[FB];
    wr[0] = frag(wrow);
#pragma unroll
    for (int f = 0; f < FB; ++f) {
      ar[f] = frag(arow + 32 * f * BK);
      sr[f] = sav[32 * f];
    }
#pragma unroll
    for (int j = 1; j < FN; ++j) wr[j] = frag(wrow + 16 * j * BK);
    const float swv = sm.sw[slot][wn >> 1];
    if (clear) {
#pragma unroll
      for (int j = 0; j < FN; ++j) clear_tail(wr[j]);
    }
    const Frag<F16> wf[FN] = {Frag<F16>(wr[0]), Frag<F16>(wr[1]), Frag<F16>(wr[2]), Frag<F16>(wr[3])};
#pragma unroll
    for (int b = 0; b < FM; b += FB) {
      if (b < nf) {
        v8i an_[FB];
        float sn[FB];
        if (b + FB < FM) {
#pragma unroll
          for (int f = 0; f < FB; ++f) {
            an_[f] = frag(arow + 32 * (b + FB + f) * BK);
            sn[f] = sav[32 * (b + FB + f)];
          }
        }
        floatx4 p[FB][FN];
#pragma unroll
        for (int f = 0; f < FB; ++f) {
          const Frag<F16> av(ar[f]);
#pragma unroll
          for (int j = 0; j < FN; ++j) p[f][j] = block_sum(wf[j], av);
        }
#pragma unroll
        for (int f = 0; f < FB; ++f) {
          const float s = sr[f] * swv;
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[b + f][j][v] = __builtin_fmaf(p[f][j][v], s, acc[b + f][j][v]);
        }
        if constexpr (!F16) {
          __builtin_amdgcn_sched_group_barrier(0x100, 6 * FB, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
#pragma unroll
          for (int t = 2; t < FB * FN; ++t) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // the FMAs of an earlier one
          }
          __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
        }
        // the sums are complete here (otherwise the compiler sinks the FMAs into
        // the next step, holding the products' registers until then)
#pragma unroll
        for (int f = 0; f < FB; ++f)
#pragma unroll
          for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[b + f][j]));
#pragma unroll
        for (int f = 0; f < FB; ++f) {
          ar[f] = an_[f];
          sr[f] = sn[f];
        }
      }
    }
  };

  // Lane (l16, g) of tile (i, j) holds tile row 32i + 16wm + l16 (the two
  // wavefront rows take alternate 16-row groups, so a partial tile splits
  // evenly), columns 16j + 4g .. +3 of the wavefront's 64.  Rows past the tile's
  // and columns past N go to buffer offsets that the range check drops, so the
  // number of store instructions is known and the next wait can leave them in
  // flight.  BF16: a lane pair's halves of two fragments' 8-column pieces are
  // exchanged first, so that a lane stores 16 bytes.  Returns the stores (0: not
  // known, the scalar path).  The accumulators are cleared.
  constexpr int kOutB = BF16OUT ? 2 : 4;
  auto epilogue = [&](const Tile& t) __attribute__((always_inline)) -> int {
    const int nf = (t.rows + 31) >> 5;   // row fragments that hold rows, for either wavefront row
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<uint8_t*>(c) + (int64_t)t.m0 * N * kOutB, (short)0, t.rows * N * kOutB, 0x00020000);
    uint32_t row_off = (uint32_t)((16 * wm + l16) * N);   // opaque: not hoisted out of the tile loop
    asm volatile("" : "+v"(row_off));
    const int n0 = t.n0 + WN * wn;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (i < nf) {
        const uint32_t ro = row_off + (uint32_t)(32 * i * N);
        if constexpr (WHOLE) {
          if constexpr (BF16OUT) {
#pragma unroll
            for (int j = 0; j < FN; j += 2) {
              const floatx4 x = acc[i][j], y = acc[i][j + 1];
              const v2u lo = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane16_swap(bf16x2_rne(x[0], x[1]), bf16x2_rne(y[0], y[1]), false, false));
              const v2u hi = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane16_swap(bf16x2_rne(x[2], x[3]), bf16x2_rne(y[2], y[3]), false, false));
              const int n = n0 + 16 * (j + (g & 1)) + 8 * (g >> 1);
              __builtin_amdgcn_raw_buffer_store_b128((v4u){lo[0], hi[0], lo[1], hi[1]}, rsrc,
                                                     n < N ? (ro + (uint32_t)n) * 2u : kOutOfRange, 0, 0);
            }
          } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              const int n = n0 + 16 * j + 4 * g;
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i][j]), rsrc,
                                                     n < N ? (ro + (uint32_t)n) * 4u : kOutOfRange, 0, 0);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const int n = n0 + 16 * j + 4 * g + v;
              const uint32_t o = n < N ? (ro + (uint32_t)n) * kOutB : kOutOfRange;
              if constexpr (BF16OUT)
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16x2_rne(acc[i][j][v], 0.0f), rsrc, o, 0, 0);
              else
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][v]), rsrc, o, 0, 0);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
    return WHOLE ? nf * (BF16OUT ? FN / 2 : FN) : 0;
  };

  // ------------------------------------------------------------ pipeline
  // Top of K-step s: its loads have landed (this wavefront's by the wait, everyone's
  // by the barrier; only stores may be in flight); the other slots, read in the step
  // before, take the loads of s + 1, which fly while this step computes.  A tile's
  // stores follow those loads in the first step of the next tile.
  int slot = 0, st = 0;
  auto begin_loads = [&](int to) __attribute__((always_inline)) {
    if (wk == nk) next_w();
    if (ak == nk) next_a();   // its map entries were loaded at least a step ago
    (void)issue_w(to);
    issue_a(to);
  };
  issue_map(an, 0);
  if (a_map) {
    wait_vmcnt(0);
    lds_barrier();
  }
  wk = ak = nk;
  begin_loads(0);
  Tile prev{0, 0, 0, 0};
  // The largest exponents() of the wavefront's scales so far; the FP8 kernel, which has no
  // register free, notes in LDS that it went past kNear (in a register: gate_up 234 us for 187;
  // the FP16 kernel with the note 1150 for 1125, 8192^3).  Without the check 185 and 1100.
  uint32_t reach = 0;
  for (int L = begin; L < end; L += step) {
    const Tile t = find(L, prev.e);
    const int nf = min(FM, (((t.rows + 15) >> 4) - wm + 1) >> 1);
    for (int kt = 0; kt < nk; ++kt) {
      wait_vmcnt(st);
      st = 0;
      lds_barrier();
      begin_loads(slot ^ 1);
      const bool clear = tail && kt == nk - 1;
      if (clear) {   // the activations' chunks past K (the weights' are cleared in registers)
        const int first = tail / 16;
        for (int i = tid; i < BM * 8; i += kThreads) {
          const int r = i >> 3, pc = i & 7;
          if ((pc ^ ((r >> 1) & 7)) >= first) *reinterpret_cast<uint4*>(sm.a[slot] + r * BK + pc * 16) = make_uint4(0, 0, 0, 0);
        }
        lds_barrier();
      }
      // this wavefront's scale products, a row in 64 to a lane
      float rs[(FM + 3) / 4];
#pragma unroll
      for (int h = 0; h < (FM + 3) / 4; ++h)
        rs[h] = sm.sa[slot][min(16 * wm + l16 + 32 * (g + 4 * h), t.rows - 1)];
      const float cs = sm.sw[slot][wn >> 1];
      if constexpr (!F16) reach = 0;
#pragma unroll
      for (int h = 0; h < (FM + 3) / 4; ++h) reach = max(reach, exponents(rs[h], cs));
      if constexpr (!F16)
        if (__builtin_amdgcn_ballot_w64(reach > kNear) != 0) sm.far[wave] = 1;
      if (kt == 0) st = epilogue(prev);   // before the first tile: no rows, nothing is written
      mma_step(slot, nf, clear);
      slot ^= 1;
    }
    prev = t;
  }
  (void)epilogue(prev);
  if (F16 ? __builtin_amdgcn_ballot_w64(reach > kNear) == 0 : sm.far[wave] == 0) return;

  wait_vmcnt(0);   // the stores of the rows that are formed once more
  far_tiles<BF16OUT, FM>(sm, begin, end, step, a, sa, a_rows, a_map, a_div, E, w, sw, N, K, c);
}

// ------------------------------------------------------------------ few rows per expert
// A workgroup takes 16 rows x 64 columns, a wavefront 16 columns over the whole of K by
// itself (so the blocks add up in the order of the other kernel).  The weights go
// straight into registers, kAhead blocks of 2 KiB a wavefront ahead of their use; the
// 16 activation rows, which every wavefront needs, and all scales pass through LDS,
// kChunk blocks of K at a time, the rows by direct loads that take no registers (through
// registers one token through 8 experts took 12 % longer).  kAhead is 8 for BF16 outputs, so a
// chunk's weights are all requested at its start, and none before (4: 78 us for 48, 128 rows over
// 128 experts of 1536 x 2048, 403 MB), and 2 for FP32 ones, where the converted fragments need
// the registers (4: 45 us for 42, 488 rows over 128 experts of 2048 x 768, 202 MB at 4.8
// TB/s, though 11.4 for 12.5 for one token).
constexpr int kRowsWaves = 4, kRowsH = 16, kChunk = 8;

// inclusive sum over the lanes up to this one
__device__ __forceinline__ int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row 0's sum to row 1, row 2's to row 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // rows 0 and 1's to rows 2 and 3
  return v;
}

// The expert and rows of m-tile tm (16 rows each, expert by expert); e < 0 past the last.
__device__ __forceinline__ void find_rows(const int32_t* __restrict__ offsets, int E, int Rc, int tm, int& e,
                                          int& m0, int& rows) {
  const int lane = lane_id();
  int before = 0;
  e = -1;
  for (int e0 = 0; e0 < E && e < 0; e0 += 4 * kWave) {
    int o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = off_at(offsets, Rc, min(e0 + q * kWave + lane, E));
    const int over = off_at(offsets, Rc, min(e0 + 4 * kWave, E));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (e >= 0) continue;
      const int next = q < 3 ? __builtin_amdgcn_readfirstlane(o[q < 3 ? q + 1 : q]) : over;
      int o1 = __shfl_down(o[q], 1, kWave);
      o1 = lane == kWave - 1 ? next : o1;
      const int nt = max(0, o1 - o[q] + kRowsH - 1) / kRowsH;
      const int incl = lane_scan(nt) + before;
      const uint64_t hit = __ballot(incl > tm);
      if (hit) {
        const int at = __ffsll((unsigned long long)hit) - 1;
        e = e0 + q * kWave + at;
        const int r0 = __builtin_amdgcn_readlane(o[q], at), first = __builtin_amdgcn_readlane(incl - nt, at);
        m0 = r0 + (tm - first) * kRowsH;
        rows = min(kRowsH, __builtin_amdgcn_readlane(o1, at) - m0);
      }
      before = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
  }
}

template <bool BF16OUT>
__global__ __launch_bounds__(kRowsWaves * 64)
void rows_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa, int a_rows,
                 const int32_t* __restrict__ a_map, int a_div, const int32_t* __restrict__ offsets, int E,
                 int Rc, const uint8_t* __restrict__ w, const float* __restrict__ sw, int N, int K,
                 void* __restrict__ c) {
  constexpr bool F16 = !BF16OUT;
  constexpr int kAhead = F16 ? 2 : 8;
  // block kb of row r: 8 chunks of 16 bytes, chunk ch at ch ^ (r / 2 mod 8) (conflict-free
  // fragment reads, see the other kernel)
  __shared__ __align__(16) uint8_t as[kChunk][kRowsH * BK];
  __shared__ float ss[kChunk][kRowsH];                   // products of the scales
  __shared__ __align__(16) int fars[kRowsWaves];         // some of them may be out of range
  const int tid = threadIdx.x, lane = lane_id(), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int e, m0 = 0, rows = 0;
  find_rows(offsets, E, Rc, blockIdx.y, e, m0, rows);
  if (e < 0) return;
  const int n0 = (blockIdx.x * kRowsWaves + wave) * 16;
  const int nk = (K + BK - 1) / BK, nnb = (N + BK - 1) / BK;

  // columns past N read the last one (never stored), chunks past K are zero
  const uint8_t* pw = w + ((int64_t)e * N + min(n0 + l16, N - 1)) * K;
  auto load = [&](int kb) __attribute__((always_inline)) -> v8i {
    const int k = kb * BK + 16 * g;
    const v4i z = {0, 0, 0, 0};
    return join(k < K ? *reinterpret_cast<const v4i*>(pw + k) : z,
                k + 64 < K ? *reinterpret_cast<const v4i*>(pw + k + 64) : z);
  };
  // source row of the workgroup's row r
  auto source = [&](int r) __attribute__((always_inline)) -> int {
    const int m = m0 + min(r, rows - 1);
    return a_map ? min(max(a_map[m], 0) / a_div, a_rows - 1) : m;
  };
  // Activations by direct-to-LDS loads of 1 KiB: rows 8h .. 8h+7 of a block, lane i row
  // 8h + i / 8, physical chunk i % 8; wavefront v takes h = v % 2 of every other block.
  // Chunks past K read the row's first of that block and are cleared in registers.
  const int srow = 8 * (wave & 1) + (lane >> 3);
  const int schunk = 16 * ((lane & 7) ^ ((srow >> 1) & 7));
  const int64_t mrow = source(srow), ms = source(tid >> 4);
  // the workgroup's 64 columns lie in one block of 128
  const float* psw = sw + ((int64_t)e * nnb + blockIdx.x * kRowsWaves * 16 / BK) * nk;
  const int tail = K & (BK - 1);

  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  bool far = false;   // the wavefront staged a scale product that may be out of range
  for (int k0 = 0; k0 < nk; k0 += kChunk) {
    const int nc = min(kChunk, nk - k0);
    const int r = tid >> 4, t = tid & 15;
    if (k0) __syncthreads();
    const float sa_v = t < nc ? sa[(int64_t)(k0 + t) * a_rows + ms] : 0.0f;
    const float sw_v = t < nc ? psw[k0 + t] : 0.0f;
    v8i wv[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (u < nc) wv[u] = load(k0 + u);
    for (int kb = wave >> 1; kb < nc; kb += 2) {
      const int k = (k0 + kb) * BK + schunk;
      lds_dma16(a + mrow * K + (k < K ? k : (k0 + kb) * BK), lds_addr(as[0]) + kb * (kRowsH * BK) + (wave & 1) * 1024);
    }
    if (t < kChunk) ss[t][r] = sa_v * sw_v;
    far |= __builtin_amdgcn_ballot_w64(exponents(sa_v, sw_v) > kNear) != 0;
    fars[wave] = far;
    __builtin_amdgcn_s_waitcnt(0x0F70);   // the direct loads have landed (and with them the first weights)
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < kChunk; ++kb) {
      if (kb < nc) {
        const uint8_t* arow = as[kb] + l16 * BK;
        v8i av = join(*reinterpret_cast<const v4i*>(arow + 16 * (g ^ (l16 >> 1))),
                      *reinterpret_cast<const v4i*>(arow + 16 * ((g + 4) ^ (l16 >> 1))));
        if (tail && k0 + kb == nk - 1) {
#pragma unroll
          for (int x = 0; x < 8; ++x) av[x] = 16 * (g + (x & 4)) < tail ? av[x] : 0;
        }
        const float sc = ss[kb][l16];
        const floatx4 p = block_sum(Frag<F16>(wv[kb % kAhead]), Frag<F16>(av));
        if (kb + kAhead < nc) wv[kb % kAhead] = load(k0 + kb + kAhead);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(p[v], sc, acc[v]);
      }
    }
  }

  const int4 f4 = *reinterpret_cast<const int4*>(fars);
  if (__builtin_amdgcn_readfirstlane(f4.x | f4.y | f4.z | f4.w)) {
    const int64_t src = source(l16);
    acc = far_sums<F16>(a + src * K, sa + src, a_rows, pw, psw, nk, K, g);
  }
  const int n = n0 + 4 * g;
  if (l16 >= rows) return;
  const int64_t at = (int64_t)(m0 + l16) * N + n;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if (n + x >= N) break;
    if constexpr (BF16OUT) static_cast<uint16_t*>(c)[at + x] = (uint16_t)bf16x2_rne(acc[x], 0.0f);
    else static_cast<float*>(c)[at + x] = acc[x];
  }
}

}  // namespace g8
}  // namespace nvfp4moe

using namespace nvfp4moe;

namespace {

int launch(const uint8_t* a, const float* sa, int64_t a_rows, const int32_t* a_map, int32_t a_div,
           const int32_t* offsets, int32_t E, int64_t R_cap, const uint8_t* w, const float* sw, int64_t N,
           int64_t K, void* c, int32_t c_dtype, void* stream) {
  if (c_dtype != NVFP4_OUT_F32 && c_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_ARG;
  if (E < 1 || E > NVFP4MOE_MAX_EXPERTS || R_cap < 0 || a_rows < 0) return NVFP4_ERR_SHAPE;
  if (K <= 0 || K % 16 != 0 || K > FP8_MAX_K || N < 1 || N > FP8_MAX_N) return NVFP4_ERR_SHAPE;
  if (R_cap > INT32_MAX / 2 || a_rows > INT32_MAX / 2) return NVFP4_ERR_SHAPE;
  // a gathered operand is addressed with 32-bit byte offsets from its base
  if (a_map && a_rows * K > (int64_t)UINT32_MAX) return NVFP4_ERR_SHAPE;
  if (R_cap == 0) return NVFP4_OK;
  if (a_rows == 0) return NVFP4_ERR_SHAPE;   // routed rows but nothing to read them from
  if (!a || !sa || !offsets || !w || !sw || !c) return NVFP4_ERR_NULL;
  if (!aligned16(a) || !aligned16(sa) || !aligned16(w) || !aligned16(sw) || !aligned16(c)) return NVFP4_ERR_ALIGN;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = c_dtype == NVFP4_OUT_BF16;
#define FP8_GEMM(KERNEL, GRID, THREADS) \
  KERNEL<<<GRID, THREADS, 0, s>>>(a, sa, (int)a_rows, a_map, a_div, offsets, E, (int)R_cap, w, sw, (int)N, (int)K, c)
  // Few rows per expert, and up to some 128 whatever their expert, leave tiles mostly empty
  // or CUs idle (us here / in tiles, BF16 out: one expert of 5120 x 2048, 128 rows 18 / 25,
  // 256 rows 27 / 26; 8 of 4096 x 2048, 192 rows 22 / 25, 256 rows 26 / 25; 128 of 1536 x 2048,
  // 1024 rows 78 / 85, 2048 rows 99 / 89.  FP32 out, 128 of 2048 x 768: 1024 rows 46 / 52,
  // 2048 rows 58 / 54).
  if (R_cap <= 128 + 8 * (int64_t)E) {
    // sum of ceil(rows / 16) over the experts is at most this
    const int64_t mt = std::min(R_cap, R_cap / g8::kRowsH + E);
    const dim3 grid((unsigned)((N + 16 * g8::kRowsWaves - 1) / (16 * g8::kRowsWaves)), (unsigned)mt);
    if (bf) FP8_GEMM(g8::rows_kernel<true>, grid, g8::kRowsWaves * 64);
    else FP8_GEMM(g8::rows_kernel<false>, grid, g8::kRowsWaves * 64);
    return launch_status();
  }
  const int64_t n_tiles = (N + g8::BN - 1) / g8::BN;
  constexpr int kFM8 = 8, kFM16 = 6;
  const int64_t max_tiles = ((R_cap + 63) / 64 + E) * n_tiles;
  if (max_tiles > INT32_MAX - 1024) return NVFP4_ERR_SHAPE;
  int64_t grid = max_tiles < 256 ? max_tiles : 256;   // one workgroup per CU, a multiple of 8
  if (grid >= 8) grid &= ~7ll;
  if (bf && N % 8 == 0) FP8_GEMM((g8::grouped_gemm_kernel<true, true, kFM8>), (unsigned)grid, g8::kThreads);
  else if (bf) FP8_GEMM((g8::grouped_gemm_kernel<true, false, kFM8>), (unsigned)grid, g8::kThreads);
  else if (N % 4 == 0) FP8_GEMM((g8::grouped_gemm_kernel<false, true, kFM16>), (unsigned)grid, g8::kThreads);
  else FP8_GEMM((g8::grouped_gemm_kernel<false, false, kFM16>), (unsigned)grid, g8::kThreads);
#undef FP8_GEMM
  return launch_status();
}

}  // namespace

extern "C" {

NVFP4MOE_API int fp8_grouped_gemm(const uint8_t* a_codes, const float* a_scales, const int32_t* expert_offsets,
                                  int32_t E, int64_t R_cap, const uint8_t* w_codes, const float* w_scales,
                                  int64_t N, int64_t K, void* c, int32_t c_dtype, void* stream) {
  return launch(a_codes, a_scales, R_cap, nullptr, 1, expert_offsets, E, R_cap, w_codes, w_scales, N, K, c,
                c_dtype, stream);
}

NVFP4MOE_API int fp8_grouped_gemm_gather(const uint8_t* a_codes, const float* a_scales, int64_t T,
                                         const int32_t* row_to_tk, int32_t k, const int32_t* expert_offsets,
                                         int32_t E, int64_t R_cap, const uint8_t* w_codes,
                                         const float* w_scales, int64_t N, int64_t K, void* c,
                                         int32_t c_dtype, void* stream) {
  if (k < 1 || k > NVFP4MOE_MAX_TOPK) return NVFP4_ERR_SHAPE;
  if (R_cap > 0 && !row_to_tk) return NVFP4_ERR_NULL;
  return launch(a_codes, a_scales, T, row_to_tk, k, expert_offsets, E, R_cap, w_codes, w_scales, N, K, c,
                c_dtype, stream);
}

}  // extern "C"
