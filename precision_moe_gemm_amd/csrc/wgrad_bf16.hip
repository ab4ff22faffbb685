// BF16 weight gradient of the grouped expert GEMM, gfx950:
//     dW_e[m][n] = sum over expert e's rows r of g[r][m] * x[r][n]
// (g the gradient of the expert GEMM's output, x its input), FP32 sums, every
// expert in one launch; an expert without rows gets zeros.  Either operand may
// be in token order, its rows then gathered through the routing map.
//
// The contraction runs over rows, and both operands are stored with the other
// dimension contiguous, so both tiles lie in LDS as [row][column] and every
// fragment is read with transposing LDS reads.  An expert has few rows for the
// size of its output (a training layer: some 256 rows for 1536 x 2048 outputs),
// so the output's bytes are what bounds it: two workgroups share a CU, and one's
// stores drain while the other loads and multiplies.
#include "fp8.h"

namespace nvfp4moe {
namespace wg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef short v8i16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __attribute__((address_space(3))) void lds_void;

// Tiles of 128 (m) x 256 (n), four wavefronts of 64 x 128, K-step 32 rows.
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

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Direct-to-LDS load of the active lanes: lane i's 16 bytes at base + voff land
// at lds + 16 i (the kernel waits itself, see gemm_bf16.hip).
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" :: "s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

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
};

// Workgroup -> (expert, tile).  Consecutive workgroups go to the 8 XCDs in turn, so
// an XCD takes whole experts, every eighth one, and their rows stay in its L2;
// fewer experts than XCDs are cut into eight runs of tiles.
__device__ __forceinline__ bool place(int wg, int E, int per, int& e, int& tile) {
  const int xcd = wg & 7, at = wg >> 3;
  if (E >= 8) {
    e = xcd + 8 * (at / per);
    tile = at % per;
    return e < E;
  }
  const int run = (E * per + 7) / 8, L = xcd * run + at;
  e = L / per;
  tile = L % per;
  return at < run && L < E * per;
}
inline int64_t grid_of(int64_t E, int64_t per) { return E >= 8 ? 8 * ((E + 7) / 8) * per : 8 * ((E * per + 7) / 8); }

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
        const uint32_t row = op.div ? (uint32_t)min(max(sm.idx[(kt * BK + k) % kIdx], 0) / op.div, op.rows - 1) : (uint32_t)k;
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

// ------------------------------------------------------------------ few tiles
// Where the outputs are too few to fill the device with large tiles, a long expert's
// chain of K-steps is what takes the time.  Tiles of 64 x 64; the workgroup's four
// wavefronts each sum every fourth K-step of the whole tile from an LDS ring of
// their own (no barrier in the loop), and the four sums are added in wavefront order
// through LDS.
namespace small {
constexpr int B = 64, kStageB = 2 * BK * B * 2, kStages = 2, kIdxS = 1024;
struct __align__(16) Smem {
  uint8_t ring[kWaves][kStages][kStageB];   // g rows, then x rows, of 32 x 64 each
  int32_t idx[kIdxS];
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
  if (gather) {
    for (int i = tid; i < min(n_rows, kIdxS); i += kThreads) sm.idx[i] = row_to_tk[r0 + i];
    __syncthreads();
  }

  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)sm.ring[wave]);
  // an instruction q holds rows 8q .. 8q+7 of an operand: lane i gives row 8q + i / 8,
  // physical chunk i % 8; rows past the expert's last are written as zeros
  auto issue = [&](int kt, int stage) __attribute__((always_inline)) -> int {
    if (kt >= nk) return 0;
    const int left = n_rows - kt * BK;
    int count = 0;
    auto one = [&](const Operand& op, int q, int c0, int cols, int at_b) __attribute__((always_inline)) {
      const int k = 8 * q + (lane >> 3);
      if (k < left) {
        const int col = min(c0 + 8 * ((lane & 7) ^ swz8(k)), cols - 8);
        const int r = kt * BK + k;
        const uint16_t* base = op.div ? op.base : op.base + (int64_t)(r0 + kt * BK) * op.ld;
        uint32_t row = (uint32_t)k;
        if (op.div) row = (uint32_t)min(max(r < kIdxS ? sm.idx[r] : row_to_tk[r0 + r], 0) / op.div, op.rows - 1);
        lds_dma16(base, (row * (uint32_t)op.ld + col) * 2u, __builtin_amdgcn_readfirstlane(lds0 + stage * kStageB + at_b + q * 1024));
      } else {
        *reinterpret_cast<uint4*>(sm.ring[wave][stage] + at_b + q * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
      }
      if (8 * q < left) ++count;
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) one(G, q, m0, M, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) one(X, q, n0, N, BK * B * 2);
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
  (void)issue(wave, 0);
  for (int kt = wave, s = 0; kt < nk; kt += kWaves, s ^= 1) {
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
  __shared__ __align__(16) float first[3][4][kWave][4];
  if (wave == 0) {
#pragma unroll
    for (int i = 1; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<floatx4*>(first[i - 1][j][lane]) = acc[i][j];
  }
  __syncthreads();
  const int m = m0 + 16 * wave + l16;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    floatx4 v = wave == 0 ? acc[0][j] : *reinterpret_cast<const floatx4*>(first[wave - 1][j][lane]);
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
  const wg::Operand G{g, (int)M, (int)g_rows, g_k}, X{x, (int)N, (int)x_rows, x_k};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = c_dtype == NVFP4_OUT_BF16;
  int64_t mt = (M + wg::BM - 1) / wg::BM, nt = (N + wg::BN - 1) / wg::BN;
  const bool few = E * mt * nt < 256;   // not one large tile per CU
  if (few) {
    mt = (M + wg::small::B - 1) / wg::small::B;
    nt = (N + wg::small::B - 1) / wg::small::B;
  }
  const int64_t grid = wg::grid_of(E, mt * nt);
  if (grid > INT32_MAX) return NVFP4_ERR_SHAPE;
#define WGRAD(KERNEL)                                                                                                 \
  KERNEL<<<(unsigned)grid, wg::kThreads, 0, s>>>(G, X, row_to_tk, expert_offsets, E, (int)R_cap, (int)M, (int)N, (int)mt, \
                                                 (int)nt, c)
  if (few) {
    if (bf) WGRAD(wg::small::grouped_wgrad_kernel<true>); else WGRAD(wg::small::grouped_wgrad_kernel<false>);
  } else {
    if (bf) WGRAD(wg::grouped_wgrad_kernel<true>); else WGRAD(wg::grouped_wgrad_kernel<false>);
  }
#undef WGRAD
  return launch_status();
}
