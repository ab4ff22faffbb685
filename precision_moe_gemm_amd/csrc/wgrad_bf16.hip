// BF16 weight gradient of the grouped expert GEMM, gfx950:
//     dW_e[m][n] = sum over expert e's rows r of g[r][m] * x[r][n]
// (g the gradient of the expert GEMM's output, x its input), FP32 sums, every
// expert in one launch; an expert without rows gets zeros.  Either operand may
// be in token order, its rows then gathered through the routing map.
//
// The contraction runs over rows, and both operands are stored with the other
// dimension contiguous, so both tiles lie in LDS as [row][column] and every
// fragment is read with transposing LDS reads.  An expert has few rows for the
// size of its output (a training layer: some 256 rows for 1536 x 2048 outputs), so
// the output's bytes are what bounds it, and how well they drain beside the loads.
// Three kernels, chosen by the number of tiles (the rule and what it measured are at
// the entry point):
//   big    256 x 256 tiles, one persistent workgroup per CU, loads running into the
//          next tile: 128 experts of 1536 x 2048 over 32768 rows, gathered, f32 out:
//          510 us (1.61 GB of output at 3.2 TB/s, 405 TFLOP/s), bf16 out 383 us.  The
//          stores overlap with neither loads nor products: a fill of the output takes 237
//          us, the loads alone 222, and it takes 457 with the products left out, 427 with
//          the loads left out, 311 with the stores left out.  All eight wavefronts issue
//          a tile's 32 stores together, on every CU at about the same time;
//   mid    128 x 256 tiles, two workgroups per CU, one's stores beside the other's
//          loads: the same 587 us, but less padding and finer balance;
//   small  64 x 64 tiles, K split over the wavefronts: one expert of 4096 rows,
//          1024 x 2048: 38 us (450 TFLOP/s; mid 142): 32 K-steps to a wavefront, their
//          loads requested one step ahead, so each pays most of a memory latency.
#include "fp8.h"
#include "lds_dma.h"

#include <algorithm>

namespace nvfp4moe {
namespace wg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

// The mid kernel.  Tiles of 128 (m) x 256 (n), four wavefronts of 64 x 128, K-step 32 rows.
constexpr int BM = 128, BN = 256, BK = 32;
constexpr int kWaves = 4, kThreads = kWaves * 64;
constexpr int FM = 4, FN = 8;
constexpr int kGB = BK * BM * 2, kXB = BK * BN * 2, kStageB = kGB + kXB;   // 8 + 16 KiB
constexpr int kStages = 3;
constexpr int kGI = kGB / 1024 / kWaves, kXI = kXB / 1024 / kWaves;        // load instructions per wavefront
constexpr int kIdx = 1024;                                                // row ids held at a time

struct __align__(16) Smem {
  uint8_t ring[kStages * kStageB];
  int32_t idx[kIdx];
};
static_assert(sizeof(Smem) <= 80 * 1024, "two workgroups per CU");

// Physical 16-byte chunk of logical chunk p of row k: p ^ swz(k).  A transposing
// read covers rows k0 .. k0+3 in each group of 16 lanes and one LDS cycle serves
// two groups, whose rows are 8 apart: the 2 (k % 4) term spreads the four rows
// over distinct banks, the 8 (k / 8 % 2) term moves the second group's to the
// other half.
__device__ __forceinline__ int swz(int k) { return (2 * (k & 3)) | (8 * ((k >> 3) & 1)); }

__device__ __forceinline__ void wait_vmcnt(int n) {
  // s_waitcnt vmcnt(n) for n up to 6 (expcnt, lgkmcnt at their maxima), else vmcnt(0)
  switch (n) {
#define WG_W(i) case i: __builtin_amdgcn_s_waitcnt(0x0F70 | i); break;
    WG_W(1) WG_W(2) WG_W(3) WG_W(4) WG_W(5) WG_W(6)
#undef WG_W
    default: __builtin_amdgcn_s_waitcnt(0x0F70); break;
  }
}

__device__ __forceinline__ int off_at(const int32_t* __restrict__ offsets, int Rc, int e) {
  return min(max(offsets[e], 0), Rc);
}

// One operand of the tile: `cols` columns of a [rows][ld] matrix from column c0,
// its rows those of the expert in order (div == 0) or row_to_tk / div.
struct Operand {
  const uint16_t* base;
  int ld, rows, div;
  uint32_t recip;   // 2^32 / div, rounded down (div 1: 2^32 - 1)
  // row of an id v of the map, kept inside the operand
  __device__ __forceinline__ uint32_t row_of(int v) const {
    // n recip / 2^32 is short of n / div by less than 1 (n < 2^31), so its integer part
    // is the quotient or one less
    const uint32_t n = (uint32_t)max(v, 0);
    uint32_t q = __umulhi(n, recip);
    q += n - q * (uint32_t)div >= (uint32_t)div;
    return min(q, (uint32_t)(rows - 1));
  }
};
inline Operand operand(const uint16_t* base, int64_t ld, int64_t rows, int div) {
  return {base, (int)ld, (int)rows, div, div ? (uint32_t)std::min<uint64_t>((1ull << 32) / div, UINT32_MAX) : 0u};
}

// Workgroup -> (expert, tile).  Consecutive workgroups go to the 8 XCDs in turn.  The
// tiles of all experts, expert by expert in the order 0, 8, 16, .., 1, 9, .., are cut
// into eight equal runs, one for each XCD: an expert's rows stay in one L2 (two where a
// cut falls inside it), and neighbouring experts, often alike in size, on different XCDs.
__device__ __forceinline__ bool place(int wg, int E, int per, int& e, int& tile) {
  const int run = (E * per + 7) / 8, at = wg >> 3, L = (wg & 7) * run + at;
  int p = L / per;
  tile = L % per;
  const int q = E / 8, longer = E % 8 * (q + 1);   // E % 8 columns of q + 1 experts, the others of q
  if (p < longer) e = p / (q + 1) + 8 * (p % (q + 1));
  else p -= longer, e = E % 8 + p / max(q, 1) + 8 * (p % max(q, 1));
  return at < run && L < E * per;
}
inline int64_t grid_of(int64_t tiles) { return (tiles + 7) / 8 * 8; }

template <bool BF16OUT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void grouped_wgrad_kernel(Operand G, Operand X, const int32_t* __restrict__ row_to_tk,
                          const int32_t* __restrict__ offsets, int E, int Rc, int M, int N, int m_tiles,
                          int n_tiles, void* __restrict__ c) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, g = lane >> 4;

  int e, tile;
  if (!place(blockIdx.x, E, m_tiles * n_tiles, e, tile)) return;
  const int m0 = tile / n_tiles * BM, n0 = tile % n_tiles * BN;
  const int r0 = __builtin_amdgcn_readfirstlane(off_at(offsets, Rc, e));
  const int n_rows = __builtin_amdgcn_readfirstlane(max(0, off_at(offsets, Rc, e + 1) - r0));
  const int nk = (n_rows + BK - 1) / BK;

  // ------------------------------------------------------------ loads
  // A 1 KiB load instruction q holds rows 4q .. 4q+3 of g (lane i: row 4q + i / 16,
  // physical chunk i % 16) or rows 2q, 2q+1 of x (row 2q + i / 32, chunk i % 32).
  // Rows past the expert's last are written as zeros by their lanes; columns past
  // the matrix read its last 8 (never stored).
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)sm.ring;
  // loads of K-step kt into its stage; returns the load instructions issued
  auto issue = [&](int kt) __attribute__((always_inline)) -> int {
    if (kt >= nk) return 0;
    const int left = n_rows - kt * BK;
    uint8_t* S = sm.ring + (kt % kStages) * kStageB;
    const uint32_t s0 = __builtin_amdgcn_readfirstlane(lds0 + (kt % kStages) * kStageB);
    int count = 0;
    auto one = [&](const Operand& op, int q, int per_q, int c0, int cols, int at_b) __attribute__((always_inline)) {
      const int lanes = 64 / per_q;
      const int k = per_q * q + lane / lanes;
      uint8_t* dst = S + at_b + q * 1024 + lane * 16;
      if (k < left) {
        const int col = min(c0 + 8 * ((lane & (lanes - 1)) ^ swz(k)), cols - 8);
        // rows in order start at the expert's first (a 64-bit base), gathered
        // ones at the operand's (the host keeps it under 4 GiB)
        const uint16_t* base = op.div ? op.base : op.base + (int64_t)(r0 + kt * BK) * op.ld;
        const uint32_t row = op.div ? op.row_of(sm.idx[(kt * BK + k) % kIdx]) : (uint32_t)k;
        lds_dma16(base, (row * (uint32_t)op.ld + col) * 2u, s0 + at_b + q * 1024);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
      }
      if (per_q * q < left) ++count;
    };
#pragma unroll
    for (int u = 0; u < kGI; ++u) one(G, wave * kGI + u, 4, m0, M, 0);
#pragma unroll
    for (int u = 0; u < kXI; ++u) one(X, wave * kXI + u, 2, n0, N, kGB);
    return count;
  };
  const bool gather = G.div || X.div;
  auto fill_idx = [&](int from) __attribute__((always_inline)) {   // row ids [from, from + kIdx)
    for (int i = tid; i < kIdx && from + i < n_rows; i += kThreads) sm.idx[(from + i) % kIdx] = row_to_tk[r0 + from + i];
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // 16 columns from `col` of a stage's [32][width] tile: lane (l16, g) receives
  // column l16 of rows 8g .. 8g+7.  In each group of 16 lanes, lane p points at
  // columns 4 (p % 4) .. +3 of row k0 + p / 4 and lane i receives column i of
  // rows k0 .. k0+3; two reads make the eight.
  auto frag = [&](const uint8_t* t, int row_b, int col) __attribute__((always_inline)) -> bf16x8 {
    v4i16 v[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int k = 8 * g + 4 * hh + (l16 >> 2);
      const int cc = col + 4 * (l16 & 3);
      v[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4i16*)(t + k * row_b + (((cc >> 3) ^ swz(k)) * 16) + ((cc >> 2) & 1) * 8));
    }
    return __builtin_bit_cast(bf16x8, (v8i16){v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]});
  };
  auto mma_step = [&](const uint8_t* S) __attribute__((always_inline)) {
    bf16x8 gv[FM], xv[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) gv[i] = frag(S, BM * 2, 64 * wm + 16 * i);
#pragma unroll
    for (int j = 0; j < FN; ++j) xv[j] = frag(S + kGB, BN * 2, 128 * wn + 16 * j);
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[j], gv[i], acc[i][j], 0, 0, 0);
  };

  // ------------------------------------------------------------ pipeline
  // At the top of K-step kt its loads have landed, those of kt + 1 may be in
  // flight; the barrier frees the stage of kt - 1, which kt + 2 then fills.
  if (gather) {
    fill_idx(0);
    __syncthreads();
  }
  issue(0);
  int next = issue(1);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vmcnt(next);
    lds_barrier();
    // the row ids of K-steps below kt + 2 are used up: the next kIdx replace them
    if (gather && kt + 2 < nk && (kt + 2) * BK % kIdx == 0) {
      fill_idx((kt + 2) * BK);
      __syncthreads();
    }
    next = issue(kt + 2);
    mma_step(sm.ring + (kt % kStages) * kStageB);
  }

  // lane (l16, g) of fragment (i, j): row m = 16i + l16, columns n = 16j + 4g .. +3
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + 64 * wm + 16 * i + l16;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int n = n0 + 128 * wn + 16 * j + 4 * g;
      if (m < M && n < N) {
        const int64_t o = ((int64_t)e * M + m) * N + n;
        const floatx4 v = acc[i][j];
        if constexpr (BF16OUT)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c) + o) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
        else
          *reinterpret_cast<floatx4*>(static_cast<float*>(c) + o) = v;
      }
    }
  }
}

// ------------------------------------------------------------------ many tiles
// Tiles of 256 x 256, a persistent workgroup of 8 wavefronts (2 x 4, 128 x 64 each) per
// CU, K-step 32 rows, a ring of four stages.  Loads run three K-steps ahead, on into
// the next tile, so a tile's stores, issued in the next tile's first step, have the
// loads of its first four steps before them and drain under those.  Measured and not
// taken: non-temporal stores (595 us for 520), stores of whole 128-byte lines by a lane
// exchange (515 us), both (594).
namespace big {
constexpr int BM = 256, BN = 256;
constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int FM = 8, FN = 4;
constexpr int kOpB = BK * 256 * 2, kStageB = 2 * kOpB;   // 16 KiB an operand
constexpr int kStages = 4;
constexpr int kIdx = 1024;                               // row ids of one run of an expert's rows
constexpr uint32_t kOutOfRange = 0x80000000u;            // buffer offset that the range check drops

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

struct __align__(16) Smem {
  uint8_t ring[kStages][kStageB];
  int32_t idx[2][kIdx];
  int off[NVFP4MOE_MAX_EXPERTS + 1];
};
static_assert(sizeof(Smem) <= 160 * 1024, "LDS");

// at most n of this wavefront's loads and stores outstanding (or fewer: n is rounded
// down to one of the counts below)
__device__ __forceinline__ void wait_vmcnt(int n) {
#define BIG_W(v) __builtin_amdgcn_s_waitcnt(0x0F70 | ((v) & 15) | ((v) >> 4 << 14))
  if (n >= 16) {
    if (n >= 40) BIG_W(40);
    else if (n >= 36) BIG_W(36);
    else if (n >= 32) BIG_W(32);
    else if (n >= 24) BIG_W(24);
    else if (n >= 20) BIG_W(20);
    else BIG_W(16);
  } else {
    if (n >= 8) BIG_W(8);
    else if (n >= 6) BIG_W(6);
    else if (n >= 4) BIG_W(4);
    else if (n >= 2) BIG_W(2);
    else BIG_W(0);
  }
#undef BIG_W
}

template <bool BF16OUT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void grouped_wgrad_kernel(Operand G, Operand X, const int32_t* __restrict__ row_to_tk,
                          const int32_t* __restrict__ offsets, int E, int Rc, int M, int N, int m_tiles,
                          int n_tiles, void* __restrict__ c) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, g = lane >> 4;
  const bool gather = G.div || X.div;
  for (int e = tid; e <= E; e += kThreads) sm.off[e] = off_at(offsets, Rc, e);
  __syncthreads();

  // The workgroup's tiles: number j is place((its XCD) + 8 (its number on the XCD + 32 j)).
  const int per = m_tiles * n_tiles;
  const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
  const int run = (E * per + 7) / 8;   // tile slots of an XCD
  struct Tile {
    int e, m0, n0, r0, rows;   // e < 0: an empty slot
  };
  auto tile_of = [&](int at) __attribute__((always_inline)) -> Tile {
    Tile t{-1, 0, 0, 0, 0};
    int e, tile;
    if (at < run && place(xcd + 8 * at, E, per, e, tile)) {
      t.e = e;
      t.m0 = tile / n_tiles * BM;
      t.n0 = tile % n_tiles * BN;
      t.r0 = __builtin_amdgcn_readfirstlane(sm.off[e]);
      t.rows = max(0, __builtin_amdgcn_readfirstlane(sm.off[e + 1]) - t.r0);
    }
    return t;
  };

  // ------------------------------------------------------------ loads
  // The cursor: K-step lk of tile lt (lat its slot; past the last slot there is none).
  // A 1 KiB instruction q of an operand holds rows 2q, 2q+1 (lane i: row 2q + i / 32,
  // physical chunk i % 32); wavefront v issues q = 2v, 2v+1 of both.
  int lat = blockIdx.x >> 3, lk = 0, lstage = 0;
  Tile lt = tile_of(lat);
  auto skip = [&]() __attribute__((always_inline)) {   // to a tile that has rows
    while (lat < run && lt.rows <= 0) {
      lat += step;
      lt = tile_of(lat);
    }
  };
  skip();
  // Row ids: run `chunk` (kIdx rows) of expert e is key e * 2^20 + chunk; idx[ib] holds
  // have, the other buffer holds (or is being filled with) ahead since `age` steps.
  int ib = 0, have = -1, ahead = -1, age = 0;
  auto fill = [&](int buf, int r0, int rows, int chunk) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kIdx / kThreads; ++u) {
      const int i = u * kThreads + wave * 64;
      if (chunk * kIdx + i < rows)
        lds_dma4(row_to_tk + r0 + chunk * kIdx, 4 * min(i + lane, rows - 1 - chunk * kIdx),
                 __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)sm.idx[0]) + (buf * kIdx + i) * 4);
    }
  };
  auto want_ids = [&]() __attribute__((always_inline)) {
    const int chunk = lk * BK / kIdx, key = (lt.e << 20) + chunk;
    if (key == have) return;
    if (key != ahead) {
      fill(ib ^ 1, lt.r0, lt.rows, chunk);
      age = 0;
    }
    if (age < kStages) {   // not yet covered by the waits of the K-loop
      __builtin_amdgcn_s_waitcnt(0x0F70);
      lds_barrier();
    }
    ib ^= 1;
    have = key;
    ahead = -1;
    // the run after this one: the expert's next, or the first of the next tile's expert
    if ((chunk + 1) * kIdx < lt.rows) {
      ahead = key + 1;
      fill(ib ^ 1, lt.r0, lt.rows, chunk + 1);
    } else {
      int at = lat + step;
      Tile n = tile_of(at);
      while (at < run && n.rows <= 0) {
        at += step;
        n = tile_of(at);
      }
      if (at < run && (n.e << 20) != have) {
        ahead = n.e << 20;
        fill(ib ^ 1, n.r0, n.rows, 0);
      }
    }
    age = 0;
  };
  auto issue = [&]() __attribute__((always_inline)) -> int {   // returns the load instructions issued
    if (lat >= run) return 0;
    if (gather) {
      want_ids();
      ++age;
    }
    const int left = lt.rows - lk * BK;
    const uint32_t s0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)sm.ring[0]) + lstage * kStageB;
    int count = 0;
    auto one = [&](const Operand& op, int q, int c0, int cols, int at_b) __attribute__((always_inline)) {
      const int k = 2 * q + (lane >> 5);
      if (k < left) {
        const int col = min(c0 + 8 * ((lane & 31) ^ swz(k)), cols - 8);
        // rows in order start at the expert's first (a 64-bit base), gathered ones at
        // the operand's (the host keeps it under 4 GiB)
        const uint16_t* base = op.div ? op.base : op.base + (int64_t)(lt.r0 + lk * BK) * op.ld;
        const uint32_t row = op.div ? op.row_of(sm.idx[ib][(lk * BK + k) % kIdx]) : (uint32_t)k;
        lds_dma16(base, (row * (uint32_t)op.ld + col) * 2u, __builtin_amdgcn_readfirstlane(s0 + at_b + q * 1024));
      } else {   // rows past the expert's last
        *reinterpret_cast<uint4*>(sm.ring[lstage] + at_b + q * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
      if (2 * q < left) ++count;
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) one(G, 2 * wave + u, lt.m0, M, 0);
#pragma unroll
    for (int u = 0; u < 2; ++u) one(X, 2 * wave + u, lt.n0, N, kOpB);
    lstage = (lstage + 1) % kStages;
    if (++lk * BK >= lt.rows) {
      lk = 0;
      lat += step;
      lt = tile_of(lat);
      skip();
    }
    return count;
  };

  floatx4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  // as in the kernel above, for rows of 512 bytes
  auto frag = [&](const uint8_t* t, int col) __attribute__((always_inline)) -> bf16x8 {
    v4i16 v[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int k = 8 * g + 4 * hh + (l16 >> 2);
      const int cc = col + 4 * (l16 & 3);
      v[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4i16*)(t + k * 512 + (((cc >> 3) ^ swz(k)) * 16) + ((cc >> 2) & 1) * 8));
    }
    return __builtin_bit_cast(bf16x8, (v8i16){v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]});
  };
  auto mma_step = [&](const uint8_t* S) __attribute__((always_inline)) {
    bf16x8 xv[FN], gv[FM];
#pragma unroll
    for (int j = 0; j < FN; ++j) xv[j] = frag(S + kOpB, 64 * wn + 16 * j);
#pragma unroll
    for (int i = 0; i < FM; ++i) gv[i] = frag(S, 128 * wm + 16 * i);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[j], gv[i], acc[i][j], 0, 0, 0);
  };
  // Lane (l16, g) of fragment (i, j): row m = 16i + l16, columns n = 16j + 4g .. +3.  Every
  // store instruction is issued (rows and columns outside go to offsets that the range
  // check drops), so that a wait can leave a known number in flight.
  constexpr int kOutB = BF16OUT ? 2 : 4, kStores = BF16OUT ? FM * FN / 2 : FM * FN;
  auto epilogue = [&](const Tile& t) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<uint8_t*>(c) + ((int64_t)t.e * M + t.m0) * N * kOutB, (short)0, min(BM, M - t.m0) * N * kOutB, 0x00020000);
    uint32_t row_off = (uint32_t)((128 * wm + l16) * N);   // opaque: not hoisted out of the tile loop
    asm volatile("" : "+v"(row_off));
    const int n0 = t.n0 + 64 * wn;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const uint32_t ro = row_off + (uint32_t)(16 * i * N);
      if constexpr (BF16OUT) {
        // a lane pair's halves of two fragments' 8-column pieces change places, so that
        // a lane stores 16 bytes
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
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    }
  };

  // ------------------------------------------------------------ pipeline
  // Top of K-step s: its loads have landed, those of s + 1 and s + 2 may be in flight;
  // the barrier frees the stage of s - 1, which the loads of s + 3 then take.  A tile's
  // stores follow the loads issued in its last step: the next three waits may leave
  // them in flight.
  int n1 = 0, n2 = 0, stores = 0, stage = 0;
#pragma unroll 1
  for (int i = 0; i < 3; ++i) {
    n1 = n2;
    n2 = issue();
  }
  for (int at = blockIdx.x >> 3; at < run; at += step) {
    const Tile t = tile_of(at);
    if (t.e < 0) continue;
    for (int kt = 0; kt * BK < t.rows; ++kt) {
      wait_vmcnt(n1 + n2 + (stores > 0 ? kStores : 0));
      --stores;
      lds_barrier();
      n1 = n2;
      n2 = issue();
      __builtin_amdgcn_sched_barrier(0);
      mma_step(sm.ring[stage]);
      stage = (stage + 1) % kStages;
      __builtin_amdgcn_sched_barrier(0);
    }
    epilogue(t);   // zeros for an expert without rows (its extra stores only make the next waits stricter)
    stores = 3;
  }
}
}  // namespace big

// ------------------------------------------------------------------ few tiles
// Where the outputs are too few to fill the device with large tiles, a long expert's
// chain of K-steps is what takes the time.  Tiles of 64 x 64; the workgroup's four
// wavefronts each sum every fourth K-step of the whole tile from an LDS ring of
// their own (no barrier in the loop), and the four sums are added in wavefront order
// through LDS.
namespace small {
constexpr int B = 64, kStageB = 2 * BK * B * 2, kStages = 2;
struct __align__(16) Smem {
  uint8_t ring[kWaves][kStages][kStageB];   // g rows, then x rows, of 32 x 64 each
  int32_t idx[kWaves][kStages][BK];         // row ids of a K-step
  float first[3][4][kWave][4];
};
static_assert(sizeof(Smem) <= 80 * 1024 && 3 * B * B * 4 <= sizeof(Smem::ring), "two workgroups per CU");

// rows of 128 bytes, two to a pass over the banks: as swz, for 8 chunks a row
__device__ __forceinline__ int swz8(int k) { return (2 * ((k >> 1) & 1)) | (4 * ((k >> 3) & 1)); }

template <bool BF16OUT>
__global__ __launch_bounds__(kThreads)
void grouped_wgrad_kernel(Operand G, Operand X, const int32_t* __restrict__ row_to_tk,
                          const int32_t* __restrict__ offsets, int E, int Rc, int M, int N, int m_tiles,
                          int n_tiles, void* __restrict__ c) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  int e, tile;
  if (!place(blockIdx.x, E, m_tiles * n_tiles, e, tile)) return;
  const int m0 = tile / n_tiles * B, n0 = tile % n_tiles * B;
  const int r0 = __builtin_amdgcn_readfirstlane(off_at(offsets, Rc, e));
  const int n_rows = __builtin_amdgcn_readfirstlane(max(0, off_at(offsets, Rc, e + 1) - r0));
  const int nk = (n_rows + BK - 1) / BK;
  const bool gather = G.div || X.div;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)sm.ring[wave]);
  // the ids of K-step kt, by lane (the upper half repeats the lower)
  const uint32_t ids0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)sm.idx[wave]);
  auto issue_ids = [&](int kt, int stage) __attribute__((always_inline)) {
    if (gather && kt < nk && lane < BK)
      lds_dma4(row_to_tk + r0 + kt * BK, 4 * min(lane, n_rows - 1 - kt * BK), ids0 + stage * BK * 4);
  };
  // an instruction q holds rows 8q .. 8q+7 of an operand: lane i gives row 8q + i / 8,
  // physical chunk i % 8; rows past the expert's last are written as zeros
  auto issue = [&](int kt, int stage) __attribute__((always_inline)) -> int {
    if (kt >= nk) return 0;
    const int left = n_rows - kt * BK;
    int count = 0;
    const int id = gather ? sm.idx[wave][stage][lane & (BK - 1)] : 0;
    // each lane works out one row's offset, the rows of an instruction take theirs from it
    const uint32_t row_g = G.div ? G.row_of(id) * (uint32_t)G.ld : 0u, row_x = X.div ? X.row_of(id) * (uint32_t)X.ld : 0u;
    auto one = [&](const Operand& op, uint32_t rows_off, int q, int c0, int cols, int at_b) __attribute__((always_inline)) {
      const int k = 8 * q + (lane >> 3);
      uint32_t off = (uint32_t)(k * op.ld);
      if (op.div) off = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * k, (int)rows_off);
      if (k < left) {
        const int col = min(c0 + 8 * ((lane & 7) ^ swz8(k)), cols - 8);
        const uint16_t* base = op.div ? op.base : op.base + (int64_t)(r0 + kt * BK) * op.ld;
        lds_dma16(base, (off + col) * 2u, __builtin_amdgcn_readfirstlane(lds0 + stage * kStageB + at_b + q * 1024));
      } else {
        *reinterpret_cast<uint4*>(sm.ring[wave][stage] + at_b + q * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
      if (8 * q < left) ++count;
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) one(G, row_g, q, m0, M, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) one(X, row_x, q, n0, N, BK * B * 2);
    return count;
  };
  auto frag = [&](const uint8_t* t, int col) __attribute__((always_inline)) -> bf16x8 {
    v4i16 v[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int k = 8 * g + 4 * hh + (l16 >> 2);
      const int cc = col + 4 * (l16 & 3);
      v[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4i16*)(t + k * (B * 2) + (((cc >> 3) ^ swz8(k)) * 16) + ((cc >> 2) & 1) * 8));
    }
    return __builtin_bit_cast(bf16x8, (v8i16){v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]});
  };
  floatx4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // this wavefront's K-steps wave, wave + 4, ..; a step's loads fly while the one before
  // it is multiplied
  issue_ids(wave, 0);
  issue_ids(wave + kWaves, 1);
  __builtin_amdgcn_s_waitcnt(0x0F70);                        // vmcnt(0)
  asm volatile("" ::: "memory");
  (void)issue(wave, 0);
  for (int kt = wave, s = 0; kt < nk; kt += kWaves, s ^= 1) {
    issue_ids(kt + 2 * kWaves, s);                           // used by the next turn's issue
    const int next = issue(kt + kWaves, s ^ 1);
    // the loads of this step have landed and the zeros are written: one wavefront's
    // own, so no barrier
    if (next == 8) __builtin_amdgcn_s_waitcnt(0x0070 | 8);   // vmcnt(8) lgkmcnt(0)
    else __builtin_amdgcn_s_waitcnt(0x0070);                 // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    asm volatile("" ::: "memory");
    const uint8_t* S = sm.ring[wave][s];
    bf16x8 gv[4], xv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) gv[i] = frag(S, 16 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) xv[j] = frag(S + BK * B * 2, 16 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[j], gv[i], acc[i][j], 0, 0, 0);
    // the stage is refilled two issues later: its reads are done by then
    __builtin_amdgcn_s_waitcnt(0xC07F);                      // lgkmcnt(0)
    asm volatile("" ::: "memory");
  }
  // the other wavefronts' sums, lane by lane
  __syncthreads();
  float* part = reinterpret_cast<float*>(sm.ring);
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<floatx4*>(part + ((((wave - 1) * 4 + i) * 4 + j) * kWave + lane) * 4) = acc[i][j];
  }
  // wavefront i stores row fragment i
  if (wave == 0) {
#pragma unroll
    for (int i = 1; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<floatx4*>(sm.first[i - 1][j][lane]) = acc[i][j];
  }
  __syncthreads();
  const int m = m0 + 16 * wave + l16;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    floatx4 v = wave == 0 ? acc[0][j] : *reinterpret_cast<const floatx4*>(sm.first[wave - 1][j][lane]);
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const floatx4 p = *reinterpret_cast<const floatx4*>(part + (((x * 4 + wave) * 4 + j) * kWave + lane) * 4);
      v += p;
    }
    const int n = n0 + 16 * j + 4 * g;
    if (m < M && n < N) {
      const int64_t o = ((int64_t)e * M + m) * N + n;
      if constexpr (BF16OUT)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c) + o) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
      else
        *reinterpret_cast<floatx4*>(static_cast<float*>(c) + o) = v;
    }
  }
}
}  // namespace small

}  // namespace wg
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" NVFP4MOE_API int bf16_grouped_gemm_wgrad(const uint16_t* g, int64_t g_rows, int32_t g_k,
                                                    const uint16_t* x, int64_t x_rows, int32_t x_k,
                                                    const int32_t* row_to_tk, const int32_t* expert_offsets,
                                                    int32_t E, int64_t R_cap, int64_t M, int64_t N, void* c,
                                                    int32_t c_dtype, void* stream) {
  if (c_dtype != NVFP4_OUT_F32 && c_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_ARG;
  if (E < 1 || E > NVFP4MOE_MAX_EXPERTS || R_cap < 0 || R_cap > INT32_MAX / 2) return NVFP4_ERR_SHAPE;
  if (M < 8 || M % 8 != 0 || M > FP8_MAX_N || N < 8 || N % 8 != 0 || N > FP8_MAX_N) return NVFP4_ERR_SHAPE;
  if (g_k < 0 || g_k > NVFP4MOE_MAX_TOPK || x_k < 0 || x_k > NVFP4MOE_MAX_TOPK) return NVFP4_ERR_SHAPE;
  if (g_rows < 0 || g_rows > INT32_MAX / 2 || x_rows < 0 || x_rows > INT32_MAX / 2) return NVFP4_ERR_SHAPE;
  // operands in the expert-grouped order hold R_cap rows; gathered ones are addressed
  // with 32-bit byte offsets
  if ((!g_k && g_rows < R_cap) || (!x_k && x_rows < R_cap)) return NVFP4_ERR_SHAPE;
  if ((g_k && g_rows * M * 2 > (int64_t)UINT32_MAX) || (x_k && x_rows * N * 2 > (int64_t)UINT32_MAX))
    return NVFP4_ERR_SHAPE;
  if (R_cap > 0 && (g_rows == 0 || x_rows == 0)) return NVFP4_ERR_SHAPE;
  if (!expert_offsets || !c || (R_cap > 0 && (!g || !x || ((g_k || x_k) && !row_to_tk)))) return NVFP4_ERR_NULL;
  if (!aligned16(g) || !aligned16(x) || !aligned16(c)) return NVFP4_ERR_ALIGN;
  const wg::Operand G = wg::operand(g, M, g_rows, g_k), X = wg::operand(x, N, x_rows, x_k);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = c_dtype == NVFP4_OUT_BF16;
  // Which kernel, by the number of tiles alone (us, f32 out; small / mid / big):
  // - not one 128 x 256 tile per CU: small.  1 expert of 4096 rows, 2048 x 2048: 83 / 143 /
  //   158; 8 of 1024 rows, 1024 x 768: 38 / 46 / 54; at 256 such tiles (32 x 512 x 512,
  //   8192 rows) 25 / 20 / 24.
  // - 256 x 256 tiles for more than half the CUs that pad no more than a quarter more than
  //   128 x 256 ones: big.  128 experts of 1536 x 2048, 32768 rows: 1012 / 543 / 490;
  //   9 of 1024 x 1024, 4096 rows (144 big tiles): 34 / 33 / 31.
  // - else mid.  8 experts of 1024 x 1024, 8192 rows (128 big tiles): 52 / 46 / 52;
  //   60 of 264 x 2048, 16384 rows (a third more padding): 106 / 64 / 78.
  int64_t mt = (M + wg::BM - 1) / wg::BM, nt = (N + wg::BN - 1) / wg::BN;
  const int64_t big_mt = (M + wg::big::BM - 1) / wg::big::BM, big_tiles = E * big_mt * nt;
  const bool few = E * mt * nt < 256;
  const bool many = !few && big_tiles > 128 && 8 * big_tiles <= 5 * (E * mt * nt);
  if (few) mt = (M + wg::small::B - 1) / wg::small::B, nt = (N + wg::small::B - 1) / wg::small::B;
  if (many) mt = big_mt;
  int64_t grid = wg::grid_of(E * mt * nt);
  if (grid > INT32_MAX) return NVFP4_ERR_SHAPE;
  if (many) grid = std::min<int64_t>(grid, 256);   // one workgroup per CU, a multiple of 8
#define WGRAD(KERNEL, THREADS)                                                                                       \
  KERNEL<<<(unsigned)grid, THREADS, 0, s>>>(G, X, row_to_tk, expert_offsets, E, (int)R_cap, (int)M, (int)N, (int)mt, \
                                            (int)nt, c)
  if (many) {
    if (bf) WGRAD(wg::big::grouped_wgrad_kernel<true>, wg::big::kThreads);
    else WGRAD(wg::big::grouped_wgrad_kernel<false>, wg::big::kThreads);
  } else if (few) {
    if (bf) WGRAD(wg::small::grouped_wgrad_kernel<true>, wg::kThreads);
    else WGRAD(wg::small::grouped_wgrad_kernel<false>, wg::kThreads);
  } else {
    if (bf) WGRAD(wg::grouped_wgrad_kernel<true>, wg::kThreads);
    else WGRAD(wg::grouped_wgrad_kernel<false>, wg::kThreads);
  }
#undef WGRAD
  return launch_status();
}
