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
#include "fp8.h"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace nvfp4moe {
namespace g8 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

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

// expert offsets clamped into [0, Rc]: malformed offsets give wrong rows but no
// access outside the buffers
__device__ __forceinline__ int off_at(const int32_t* __restrict__ offsets, int Rc, int e) {
  return min(max(offsets[e], 0), Rc);
}

// ------------------------------------------------------------------ many rows per expert
// A workgroup of 8 wavefronts (2 x 4) computes up to BM x 256, a wavefront up to
// 16 FM x 64 of it; the FP16 fragments of its 64 columns take 64 registers, so that
// kernel's tiles are 192 rows high, the FP8 kernel's 256.
constexpr int BN = 256, BK = kFp8Block;
constexpr int kNumHeights = 4;
constexpr int kTileCost = 96;                  // rows' worth of a tile's cost that does not scale with its rows
constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int FN = 4, WN = 64;
constexpr int kWI = BN / 8 / kWaves;           // weight load instructions per wavefront and K-step (8 rows each)
constexpr int kStages = 2;

template <bool F16>
struct Shape {
  static constexpr int FM = F16 ? 6 : 8, BM = 32 * FM;
  static constexpr int kAI = BM / 8 / kWaves;             // activation load instructions per wavefront
  static constexpr int kStageS = (BM + BN) * BK;          // scales follow the two operand tiles
  static constexpr int kSaB = (BM * 4 + 255) & ~255;
  static constexpr int kStageB = kStageS + kSaB + 256;
  // tile heights to choose from, all multiples of 32
  __host__ __device__ static constexpr int height(int i) { return i == 0 ? BM : i == 1 ? 3 * BM / 4 & ~31 : i == 2 ? 128 : 64; }
};

template <bool F16>
struct __align__(16) Smem {
  uint8_t ring[kStages * Shape<F16>::kStageB];
  int tile_start[NVFP4MOE_MAX_EXPERTS + 1];
};
static_assert(sizeof(Smem<false>) <= 160 * 1024 && sizeof(Smem<true>) <= 160 * 1024, "LDS");

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Direct-to-LDS loads: lane i's 16 (4) bytes at base + voff land at lds + 16 (4) i.
// Issued through inline assembly so that the compiler does not make every later
// LDS read wait for them; the kernel waits itself (vmcnt).
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" :: "s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" :: "s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// fn(std::integral_constant<int, v>) for the v in Is... equal to n
template <int... Is, typename Fn>
__device__ __forceinline__ void dispatch_count(int n, std::integer_sequence<int, Is...>, Fn&& fn) {
  (void)((n == Is ? (fn(std::integral_constant<int, Is>{}), true) : false) || ...);
}

struct Tile {
  int e, m0, rows, n0;
};

__device__ __forceinline__ Tile tile_at(int L, int n_tiles, const int* tile_start, int E,
                                        const int32_t* __restrict__ offsets, int Rc) {
  const int tm = L / n_tiles, tn = L - tm * n_tiles;
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= tm) lo = mid; else hi = mid;
  }
  Tile t;
  t.e = __builtin_amdgcn_readfirstlane(lo);
  // the expert's rows split evenly over its m-tiles, in 16-row groups (no tile
  // is empty, none taller than the launch's height)
  const int o0 = off_at(offsets, Rc, t.e), o1 = off_at(offsets, Rc, t.e + 1);
  const int nt = tile_start[t.e + 1] - tile_start[t.e];
  const int per = ((o1 - o0 + nt - 1) / nt + 15) & ~15;
  t.m0 = __builtin_amdgcn_readfirstlane(o0 + (tm - tile_start[t.e]) * per);
  t.rows = __builtin_amdgcn_readfirstlane(max(0, min(per, o1 - t.m0)));
  t.n0 = __builtin_amdgcn_readfirstlane(tn * BN);
  return t;
}

template <bool BF16OUT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void grouped_gemm_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa, int a_rows,
                         const int32_t* __restrict__ a_map, int a_div,
                         const int32_t* __restrict__ offsets, int E, int Rc,
                         const uint8_t* __restrict__ w, const float* __restrict__ sw, int N, int K,
                         void* __restrict__ c) {
  constexpr bool F16 = !BF16OUT;
  using S = Shape<F16>;
  constexpr int FM = S::FM, BM = S::BM, kAI = S::kAI, kStageS = S::kStageS, kStageB = S::kStageB;
  __shared__ Smem<F16> sm;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, g = lane >> 4;
  const int n_tiles = (N + BN - 1) / BN;

  if (wave == 0) {
    // Tile height: the candidate with the smallest estimated critical path,
    // (tiles per workgroup) x (height + kTileCost).  Ties go to the taller.
    const int G = gridDim.x, xg = (G & 7) == 0 ? 8 : 1;
    int best = BM;
    int64_t best_cost = INT64_MAX;
#pragma unroll
    for (int q = 0; q < kNumHeights; ++q) {
      const int h = S::height(q);
      int mt = 0;
      for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = e0 + lane;
        int v = e < E ? max(0, off_at(offsets, Rc, e + 1) - off_at(offsets, Rc, e) + h - 1) / h : 0;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
        mt += v;
      }
      const int64_t total = (int64_t)mt * n_tiles;
      const int64_t per = (total + xg - 1) / xg, wgs = G / xg;
      const int64_t cost = (per + wgs - 1) / wgs * (h + kTileCost);
      if (cost < best_cost) {
        best_cost = cost;
        best = h;
      }
    }
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += kWave) {
      const int e = e0 + lane;
      const int v = e < E ? max(0, off_at(offsets, Rc, e + 1) - off_at(offsets, Rc, e) + best - 1) / best : 0;
      int incl = v;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int y = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += y;
      }
      if (e < E) sm.tile_start[e] = carry + incl - v;
      carry += __shfl(incl, kWave - 1, kWave);
    }
    if (lane == 0) sm.tile_start[E] = carry;
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

  // ------------------------------------------------------------ load cursor
  // (lL, lk): the next K-step to load.  A load instruction q of an operand fills
  // 1 KiB, rows 8q .. 8q+7: lane i gives row 8q + i / 8, physical 16-byte chunk
  // i % 8, which holds logical chunk (i % 8) ^ (row / 2 mod 8) (see mma_step).
  // Wavefront v takes q = v, v + 8, ..; its lanes' logical chunk is the same in
  // all of them.  The first kSaWaves wavefronts also load the scales of 64 rows
  // each, the next one those of the tile's two weight column blocks.
  constexpr int kSaWaves = S::kSaB / 256;
  int lL = begin, lk = 0, l_rows = 0, l_cols = 0;
  const uint8_t *pa = nullptr, *pw = nullptr;
  const float* ps = nullptr;
  uint32_t off_a[kAI], off_w[kWI], off_s = 0;
  const int chunk = 16 * ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7));
  // the last K-step's chunks past K read the row's first chunk of that step
  // instead (in bounds); the compute side clears them
  const uint32_t back = tail && chunk >= tail ? chunk : 0;
  auto set_load_tile = [&](int L) __attribute__((always_inline)) {
    const Tile t = tile_at(L, n_tiles, sm.tile_start, E, offsets, Rc);
    l_rows = t.rows;
    l_cols = min(BN, N - t.n0);
    // gathered operand: routed row m reads row a_map[m] / a_div of a, clamped
    // into a (an invalid map entry reads a wrong row, never outside)
    auto src = [&](int r) __attribute__((always_inline)) -> uint32_t {
      const int m = min(r, t.rows - 1);
      return a_map ? (uint32_t)min(max(a_map[t.m0 + m], 0) / a_div, a_rows - 1) : (uint32_t)m;
    };
#pragma unroll
    for (int u = 0; u < kAI; ++u) off_a[u] = src(8 * (wave + kWaves * u) + (lane >> 3)) * (uint32_t)K + chunk;
#pragma unroll
    for (int u = 0; u < kWI; ++u)
      off_w[u] = (uint32_t)min(8 * (wave + kWaves * u) + (lane >> 3), l_cols - 1) * (uint32_t)K + chunk;
    pa = a_map ? a : a + (int64_t)t.m0 * K;
    pw = w + ((int64_t)t.e * N + t.n0) * K;
    if (wave < kSaWaves) {
      ps = a_map ? sa : sa + t.m0;
      off_s = 4 * src(64 * wave + lane);
    } else {
      const int nb = t.n0 / BK;
      ps = sw + ((int64_t)t.e * nnb + nb) * nk;
      off_s = 4 * nk * min(min(lane, 1), nnb - 1 - nb);
    }
  };
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)sm.ring;
  auto issue_loads = [&](int stage) __attribute__((always_inline)) {
    if (lL >= end) return;
    const uint32_t s0 = __builtin_amdgcn_readfirstlane(lds0 + stage * kStageB);
    const uint32_t bk = lk == nk - 1 ? back : 0;
#pragma unroll
    for (int u = 0; u < kAI; ++u)
      if (8 * (wave + kWaves * u) < l_rows) lds_dma16(pa, off_a[u] - bk, s0 + (wave + kWaves * u) * 1024);
#pragma unroll
    for (int u = 0; u < kWI; ++u)
      if (8 * (wave + kWaves * u) < l_cols) lds_dma16(pw, off_w[u] - bk, s0 + BM * BK + (wave + kWaves * u) * 1024);
    if (wave < kSaWaves ? 64 * wave < l_rows : wave == kSaWaves) lds_dma4(ps, off_s, s0 + kStageS + wave * 256);
    pa += BK;
    pw += BK;
    ps += wave < kSaWaves ? a_rows : 1;
    if (++lk == nk) {
      lk = 0;
      lL += step;
      if (lL < end) set_load_tile(lL);
    }
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // One K-step over the wavefront's first NF row fragments.  A fragment read
  // gives lane (l16, g) the chunks g and g + 4 of row l16 of the fragment, each
  // at its row's physical place, chunk ^ (row / 2 mod 8): a 16-byte LDS read is
  // served 16 lanes at a time, here 16 rows with chunk g from one half and
  // g ^ 1 from the other, and the XOR puts those on 16 different bank groups.
  const int pc0 = 16 * (g ^ (l16 >> 1)), pc1 = 16 * ((g + 4) ^ (l16 >> 1));
  auto frag = [&](const uint8_t* row) __attribute__((always_inline)) -> v8i {
    return join(*reinterpret_cast<const v4i*>(row + pc0), *reinterpret_cast<const v4i*>(row + pc1));
  };
  auto mma_step = [&](auto nf_tag, int stage) __attribute__((always_inline)) {
    constexpr int NF = decltype(nf_tag)::value;
    if constexpr (NF > 0) {
      const uint8_t* st = sm.ring + stage * kStageB;
      const float* scales = reinterpret_cast<const float*>(st + kStageS);
      const float swv = scales[S::kSaB / 4 + (wn >> 1)];
      const uint8_t* wrow = st + (BM + WN * wn + l16) * BK;
      const Frag<F16> wf[FN] = {Frag<F16>(frag(wrow)), Frag<F16>(frag(wrow + 16 * BK)), Frag<F16>(frag(wrow + 32 * BK)),
                                Frag<F16>(frag(wrow + 48 * BK))};
      floatx4 p[FN];
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i <= NF; ++i) {
        floatx4 q[FN];
        float sn = 0.0f;
        if (i < NF) {
          const int r = 32 * i + 16 * wm + l16;
          const Frag<F16> av(frag(st + r * BK));
          sn = scales[r] * swv;
#pragma unroll
          for (int j = 0; j < FN; ++j) q[j] = block_sum(wf[j], av);
        }
        if (i > 0) {
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i - 1][j][v] = __builtin_fmaf(p[j][v], s, acc[i - 1][j][v]);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) p[j] = q[j];
        s = sn;
      }
    }
  };

  // Lane (l16, g) of tile (i, j) holds tile row 32i + 16wm + l16 (the two
  // wavefront rows take alternate 16-row groups, so a partial tile splits
  // evenly), columns 16j + 4g .. +3 of the wavefront's 64.  Rows past the tile's
  // and columns past N are not written.  The accumulators are cleared.
  const bool whole4 = (N & 3) == 0;
  auto epilogue = [&](const Tile& t) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int r = 32 * i + 16 * wm + l16;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = t.n0 + WN * wn + 16 * j + 4 * g;
        const int64_t at = (int64_t)(t.m0 + r) * N + n;
        if (r < t.rows && n < N) {
          const floatx4 v = acc[i][j];
          if constexpr (BF16OUT) {
            uint16_t* p = static_cast<uint16_t*>(c) + at;
            const uint32_t lo = bf16x2_rne(v[0], v[1]), hi = bf16x2_rne(v[2], v[3]);
            if (whole4) {
              *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
            } else {
              p[0] = (uint16_t)lo;
              if (n + 1 < N) p[1] = (uint16_t)(lo >> 16);
              if (n + 2 < N) p[2] = (uint16_t)hi;
              if (n + 3 < N) p[3] = (uint16_t)(hi >> 16);
            }
          } else {
            float* p = static_cast<float*>(c) + at;
            if (whole4) {
              *reinterpret_cast<floatx4*>(p) = v;
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (n + x < N) p[x] = v[x];
            }
          }
        }
        acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
    }
  };

  // ------------------------------------------------------------ pipeline
  // At the top of a K-step its loads have landed (this wavefront's by the wait,
  // everyone's by the barrier); the other stage, read in the step before, takes
  // the next step's loads, which fly while this step computes.
  set_load_tile(begin);
  issue_loads(0);
  int sc = 0;
  auto top = [&](int kt) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    lds_barrier();
    issue_loads(sc ^ 1);
    if (tail && kt == nk - 1) {
      // clear the chunks past K of both operands (the other stage is untouched)
      const int first = tail / 16;
      for (int i = tid; i < (BM + BN) * 8; i += kThreads) {
        const int r = i >> 3, pc = i & 7;
        if ((pc ^ ((r >> 1) & 7)) >= first)
          *reinterpret_cast<uint4*>(sm.ring + sc * kStageB + r * BK + pc * 16) = make_uint4(0, 0, 0, 0);
      }
      lds_barrier();
    }
  };
  auto run_tile = [&](auto nf_tag) __attribute__((always_inline)) {
    mma_step(nf_tag, sc);   // K-step 0: its top is done by the caller
    sc ^= 1;
    for (int kt = 1; kt < nk; ++kt) {
      top(kt);
      mma_step(nf_tag, sc);
      sc ^= 1;
    }
  };
  Tile prev{0, 0, 0, 0};
  for (int L = begin; L < end; L += step) {
    const Tile t = tile_at(L, n_tiles, sm.tile_start, E, offsets, Rc);
    top(0);
    epilogue(prev);   // before the first tile: no rows, nothing is written
    const int nf = min(FM, (((t.rows + 15) >> 4) - wm + 1) >> 1);
    dispatch_count(nf, std::make_integer_sequence<int, FM + 1>{},
                   [&](auto nf_tag) __attribute__((always_inline)) { run_tile(nf_tag); });
    prev = t;
  }
  epilogue(prev);
}

// ------------------------------------------------------------------ few rows per expert
// A wavefront computes 16 rows x 16 columns over the whole of K by itself (so the
// blocks add up in the order of the other kernel), a workgroup 16 rows x 64
// columns.  Weights, activations and scales go straight into registers; the
// loads of kAhead blocks are issued before the first is used, 2 KiB of weights
// per wavefront and block.
constexpr int kRowsWaves = 4, kRowsN = 16 * kRowsWaves, kRowsH = 16, kAhead = 8;

template <bool BF16OUT>
__global__ __launch_bounds__(kRowsWaves * 64)
void rows_kernel(const uint8_t* __restrict__ a, const float* __restrict__ sa, int a_rows,
                 const int32_t* __restrict__ a_map, int a_div, const int32_t* __restrict__ offsets, int E,
                 int Rc, const uint8_t* __restrict__ w, const float* __restrict__ sw, int N, int K,
                 void* __restrict__ c) {
  constexpr bool F16 = !BF16OUT;
  const int lane = lane_id(), l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int tm = blockIdx.y, n0 = (blockIdx.x * kRowsWaves + wave) * 16;
  if (n0 >= N) return;

  // the expert of m-tile tm: every wavefront scans the experts, 64 at a time
  int e = -1, m0 = 0, rows = 0, before = 0;
  for (int e0 = 0; e0 < E && e < 0; e0 += kWave) {
    const int x = e0 + lane;
    const int o0 = x < E ? off_at(offsets, Rc, x) : 0, o1 = x < E ? off_at(offsets, Rc, x + 1) : 0;
    const int nt = max(0, o1 - o0 + kRowsH - 1) / kRowsH;
    int incl = nt;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int y = __shfl_up(incl, off, kWave);
      if (lane >= off) incl += y;
    }
    incl += before;
    const uint64_t hit = __ballot(incl > tm);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      const int first = __shfl(incl - nt, at, kWave), r0 = __shfl(o0, at, kWave), r1 = __shfl(o1, at, kWave);
      e = e0 + at;
      m0 = r0 + (tm - first) * kRowsH;
      rows = min(kRowsH, r1 - m0);
    }
    before = __shfl(incl, kWave - 1, kWave);
  }
  if (e < 0) return;
  e = __builtin_amdgcn_readfirstlane(e);
  m0 = __builtin_amdgcn_readfirstlane(m0);
  rows = __builtin_amdgcn_readfirstlane(rows);

  const int nk = (K + BK - 1) / BK, nnb = (N + BK - 1) / BK;
  int m = m0 + min(l16, rows - 1);
  if (a_map) m = min(max(a_map[m], 0) / a_div, a_rows - 1);
  const uint8_t* pa = a + (int64_t)m * K;
  const uint8_t* pw = w + ((int64_t)e * N + min(n0 + l16, N - 1)) * K;
  const float* psa = sa + m;
  const float* psw = sw + ((int64_t)e * nnb + n0 / BK) * nk;   // 16 columns lie in one block

  // chunks g and g + 4 of block kb of a row; chunks past K are zero
  auto load = [&](const uint8_t* row, int kb) __attribute__((always_inline)) -> v8i {
    const int k = kb * BK + 16 * g;
    const v4i z = {0, 0, 0, 0};
    return join(k < K ? *reinterpret_cast<const v4i*>(row + k) : z,
                k + 64 < K ? *reinterpret_cast<const v4i*>(row + k + 64) : z);
  };
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  auto chunk = [&](int kb0, auto full) __attribute__((always_inline)) {
    v8i wv[kAhead], av[kAhead];
    float ss[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (full || kb0 + u < nk) {
        wv[u] = load(pw, kb0 + u);
        av[u] = load(pa, kb0 + u);
        ss[u] = psa[(int64_t)(kb0 + u) * a_rows] * psw[kb0 + u];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (full || kb0 + u < nk) {
        const floatx4 p = block_sum(Frag<F16>(wv[u]), Frag<F16>(av[u]));
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(p[v], ss[u], acc[v]);
      }
    }
  };
  int kb = 0;
  for (; kb + kAhead <= nk; kb += kAhead) chunk(kb, std::true_type{});
  if (kb < nk) chunk(kb, std::false_type{});

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
#define FP8_GEMM(KERNEL, GRID, THREADS)                                                                       \
  (bf ? KERNEL<true><<<GRID, THREADS, 0, s>>>(a, sa, (int)a_rows, a_map, a_div, offsets, E, (int)R_cap, w, sw, \
                                              (int)N, (int)K, c)                                              \
      : KERNEL<false><<<GRID, THREADS, 0, s>>>(a, sa, (int)a_rows, a_map, a_div, offsets, E, (int)R_cap, w, sw, \
                                               (int)N, (int)K, c))
  if (R_cap <= 16 * (int64_t)E || R_cap <= 64) {
    // sum of ceil(rows / 16) over the experts is at most this
    const int64_t mt = std::min(R_cap, R_cap / g8::kRowsH + E);
    const dim3 grid((unsigned)((N + g8::kRowsN - 1) / g8::kRowsN), (unsigned)mt);
    FP8_GEMM(g8::rows_kernel, grid, g8::kRowsWaves * 64);
    return launch_status();
  }
  const int64_t n_tiles = (N + g8::BN - 1) / g8::BN;
  const int64_t min_h = g8::Shape<false>::height(g8::kNumHeights - 1);
  const int64_t max_tiles = ((R_cap + min_h - 1) / min_h + E) * n_tiles;
  if (max_tiles > INT32_MAX) return NVFP4_ERR_SHAPE;
  int64_t grid = max_tiles < 256 ? max_tiles : 256;   // one workgroup per CU, a multiple of 8
  if (grid >= 8) grid &= ~7ll;
  FP8_GEMM(g8::grouped_gemm_kernel, (unsigned)grid, g8::kThreads);
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
