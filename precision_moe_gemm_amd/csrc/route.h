// Routing of (token, slot) entries to expert-grouped rows, shared by the passes that permute token rows:
// ranks within chunks of the routing list, and the scan of long count tables.
#pragma once

#include "common.h"

namespace nvfp4moe {

// workgroup barrier for LDS only: global loads in flight are not waited for
__device__ __forceinline__ void lds_only_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The rank pass: workgroup c (16 wavefronts) takes chunk c of 2^L routing
// entries (L = 11 or 12, chosen per launch by plan_chunk_log).  Each
// wavefront ranks its 2^L / 16 entries in passes of 64 consecutive ones by
// ballot matching on the expert id, keeping a running count per expert in
// LDS; an exclusive scan of those counts over the wavefronts gives every entry
// its stable rank among the chunk's entries of its expert (entry order: token,
// then slot).  The ranks go to the workspace and the chunk's counts per expert
// to the table, cnt[c][e].  Workgroups are independent; the launch boundary
// publishes the results.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanChunkLogMin = 11;     // 2048 routing entries per chunk: two passes per wavefront
constexpr int kPlanChunkLogMax = 12;     // 4096: four passes
constexpr int kCountTable = 4096;        // ints of (chunk, expert) counts the main pass scans

inline int plan_chunks(int64_t n, int lg) { return n > 0 ? (int)((n + (1ll << lg) - 1) >> lg) : 1; }

// The smallest chunk whose count table still fits the main pass (more
// workgroups share the ranking of a short list), else the largest.  (At 4096
// tokens x 8 of 128 experts, chunks of 2048 entries measured best: 1024 gives
// each main-pass workgroup a 4096-int table to scan, 4096 leaves the rank pass
// on 8 workgroups.)
inline int plan_chunk_log(int64_t n, int E) {
  for (int lg = kPlanChunkLogMin; lg < kPlanChunkLogMax; ++lg)
    if ((int64_t)plan_chunks(n, lg) * E <= kCountTable) return lg;
  return kPlanChunkLogMax;
}

static __global__ __launch_bounds__(kPlanThreads) void route_rank_kernel(
    const int32_t* __restrict__ ids, int n, int E, int chunk_log, int32_t* __restrict__ cnt_out,
    int32_t* __restrict__ rank_out, int32_t* __restrict__ dev_err) {
  __shared__ int32_t wcnt[kPlanWaves][NVFP4MOE_MAX_EXPERTS];   // per wavefront, then its exclusive prefix
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const int passes = (1 << chunk_log) / kPlanThreads;           // passes of 64 per wavefront (<= 4)
  const int base = (blockIdx.x << chunk_log) + wave * 64 * passes;   // this wavefront's entries
  int ev[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = base + 64 * u + lane;
    ev[u] = (u < passes && i < n) ? ids[i] : -1;
  }
  for (int e = lane; e < E; e += kWave) wcnt[wave][e] = 0;   // each wavefront clears its own row
  const int nbits = E > 1 ? 32 - __clz(E - 1) : 0;
  const uint64_t lt_mask = (lane == 0) ? 0ull : (~0ull >> (kWave - lane));
  int lr[4] = {-1, -1, -1, -1};
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u >= passes) break;
    const int i = base + 64 * u + lane;
    const int e = ev[u];
    const bool valid = i < n && e >= 0 && e < E;
    bad |= i < n && !valid;
    uint64_t peers = __ballot(valid);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = valid && ((e >> b) & 1);
      const uint64_t bb = __ballot(bit);
      peers &= bit ? bb : ~bb;
    }
    lr[u] = -1;
    if (valid) {
      const int r = __popcll(peers & lt_mask);
      const int before = wcnt[wave][e];
      lr[u] = before + r;
      if (r == 0) wcnt[wave][e] = before + __popcll(peers);
    }
  }
  if (bad && dev_err) atomicOr(dev_err, NVFP4_DEVERR_BAD_EXPERT);
  __syncthreads();
  // exclusive scan over the wavefronts, per expert; the chunk's counts
  for (int e = tid; e < E; e += kPlanThreads) {
    int acc = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      const int v = wcnt[w][e];
      wcnt[w][e] = acc;
      acc += v;
    }
    cnt_out[blockIdx.x * E + e] = acc;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = base + 64 * u + lane;
    if (u < passes && i < n) rank_out[i] = lr[u] >= 0 ? wcnt[wave][ev[u]] + lr[u] : -1;
  }
}

// Long routing lists (a count table too large for every workgroup of the
// main pass to scan), long rows, or no tokens: the ranks as above, then one
// workgroup turns the table into first rows,
//   base[c][e] = offsets[e] + (entries of e in chunks before c),
// in place and writes the offsets; the main pass then needs no scan at all.
static __global__ __launch_bounds__(kPlanThreads) void route_scan_kernel(
    int32_t* __restrict__ table, int nchunks, int E, int32_t* __restrict__ offsets) {
  __shared__ int32_t part[kPlanThreads];
  __shared__ int32_t wsum[kPlanWaves];
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  // thread (e, p), P = 1024 / E threads per expert, sums chunks [p cpt, (p + 1) cpt)
  const int P = kPlanThreads / E, cpt = (nchunks + P - 1) / P;
  const int e = tid / P, p = tid - e * P;
  const int c_lo = min(nchunks, p * cpt), c_hi = min(nchunks, (p + 1) * cpt);
  int sum = 0;
  if (e < E)
    for (int c = c_lo; c < c_hi; ++c) sum += table[(int64_t)c * E + e];
  part[tid] = sum;
  __syncthreads();
  int pre_p = 0, tot = 0;
  if (e < E) {
    for (int q = 0; q < P; ++q) {
      const int v = part[e * P + q];
      if (q < p) pre_p += v;
      tot += v;
    }
  }
  // offsets: exclusive scan over experts of the totals, carried by thread (e, 0)
  const int mine = (e < E && p == 0) ? tot : 0;
  int incl = mine;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int y = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += y;
  }
  if (lane == kWave - 1) wsum[wave] = incl;
  __syncthreads();   // also: every read of part[] above is done
  int wbefore = 0;
  for (int w = 0; w < wave; ++w) wbefore += wsum[w];
  if (e < E && p == 0) part[e] = wbefore + incl - mine;
  __syncthreads();
  if (e < E) {
    const int off_e = part[e];
    if (p == 0) offsets[e] = off_e;
    int acc = off_e + pre_p;
    for (int c = c_lo; c < c_hi; ++c) {
      const int64_t at = (int64_t)c * E + e;
      const int v = table[at];
      table[at] = acc;
      acc += v;
    }
  }
  if (tid == kPlanThreads - 1) offsets[E] = wbefore + incl;
}

// What a main pass of 512-thread workgroups, each owning kRouteTokens consecutive tokens, makes of the count
// table: load() issues the table's loads (unconditional, indices clamped into it), scan() turns it into the
// expert offsets (written by workgroup 0) and, in LDS, the first row of every expert in the chunk of the
// workgroup's first entry and in the next one; its barriers order LDS alone, so that loads issued in between
// stay in flight.  Needs nchunks * E <= kCountTable.
constexpr int kRouteTokens = 8;
constexpr int kRouteThreads = 512;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kRouteExp = NVFP4MOE_MAX_EXPERTS / kRouteThreads;   // experts per thread (2)
static_assert(kRouteTokens * NVFP4MOE_MAX_TOPK <= 1 << kPlanChunkLogMin, "a workgroup's entries lie in at most two chunks");

struct RouteLds {
  int32_t first[2][NVFP4MOE_MAX_EXPERTS];   // first row of expert e in chunk c0, c0 + 1
  int32_t wsum[kRouteWaves];
  int32_t tab[kCountTable];
};

struct RouteTable {
  int tv[kCountTable / kRouteThreads];      // 8 independent loads per thread
  int c0;                                   // the chunk of the workgroup's first entry

  __device__ __forceinline__ void load(const int32_t* __restrict__ cnt, int ntab) {
#pragma unroll
    for (int u = 0; u < kCountTable / kRouteThreads; ++u)
      tv[u] = cnt[min(u * kRouteThreads + (int)threadIdx.x, ntab - 1)];
  }

  __device__ __forceinline__ void scan(RouteLds& s, int nchunks, int E, int32_t* __restrict__ offsets) {
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, ntab = nchunks * E;
#pragma unroll
    for (int u = 0; u < kCountTable / kRouteThreads; ++u) {
      const int i = u * kRouteThreads + tid;
      s.tab[i] = i < ntab ? tv[u] : 0;
    }
    lds_only_barrier();
    int tot[kRouteExp], b0[kRouteExp], b1[kRouteExp];
#pragma unroll
    for (int u = 0; u < kRouteExp; ++u) { tot[u] = 0; b0[u] = 0; b1[u] = 0; }
    for (int c = 0; c < nchunks; ++c) {
#pragma unroll
      for (int u = 0; u < kRouteExp; ++u) {
        const int e = kRouteExp * tid + u;
        const int v = e < E ? s.tab[c * E + e] : 0;
        tot[u] += v;
        if (c < c0) b0[u] += v;
        if (c <= c0) b1[u] += v;
      }
    }
    // expert offsets: exclusive scan of the totals over experts
    int mine_tot = 0;
#pragma unroll
    for (int u = 0; u < kRouteExp; ++u) mine_tot += tot[u];
    int incl = mine_tot;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int y = __shfl_up(incl, off, kWave);
      if (lane >= off) incl += y;
    }
    if (lane == kWave - 1) s.wsum[wave] = incl;
    lds_only_barrier();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += s.wsum[w];
    int off_e = before + incl - mine_tot;   // offset of expert kRouteExp * tid
#pragma unroll
    for (int u = 0; u < kRouteExp; ++u) {
      const int e = kRouteExp * tid + u;
      if (e < E) {
        s.first[0][e] = off_e + b0[u];
        s.first[1][e] = off_e + b1[u];
        if (blockIdx.x == 0) offsets[e] = off_e;
      }
      off_e += tot[u];
    }
    if (blockIdx.x == 0 && tid == kRouteThreads - 1) offsets[E] = before + incl;
    lds_only_barrier();
  }
};

}  // namespace nvfp4moe
