// gqa_kv_evict: which rows stay, and the moves that close the cache up.
//
// A row's rank is a 32-bit key, the larger the better: held rows all ones,
// others their score mapped to an order-preserving integer (NaN 0). The rows
// that stay are the `keep` largest keys, the lower row first among equal ones:
// those above the keep-th largest key tau, and the first need_eq rows equal to
// it. tau comes from a radix select, 11 + 11 + 10 bits from the top.
//
//   evict_select_kernel  a cluster of CTAs per (b, g), each with a contiguous
//     segment of the rows, whose keys it reads once and keeps in shared memory
//     (S_max 131072: 8 CTAs of 64 KB). The three histograms are summed over
//     the cluster through distributed shared memory. Then the holes (rows
//     below keep that go) and the movers (rows from keep on that stay) are
//     numbered in order of their rows: mover i goes to hole i. The scores and
//     positions move here; the rows themselves (their numbers are written to
//     the workspace) in
//   evict_move_kernel    all CTAs of the GPU, one warp per row: sources lie
//     at or above keep and destinations below it, so no order is needed.
//
// Bytes: 8 per row read (score, position), and the moved rows twice.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"

namespace gqa {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvMaxCluster = 8;
constexpr int kEvStaticBytes = (kEvBins + 4 * kEvWarps + 16) * 4;
// keys of a segment kept in shared memory; rows past these (caches of more than 8 x 40960 rows) are read again
constexpr int kEvMaxSegKeys = 40960;

struct EvictParams {
  void *k_cache, *v_cache;
  float* scores;
  int32_t* row_pos;  // or null
  int32_t* seqlens;
  const int32_t* recent_from;  // or null
  int32_t* ws;                 // per unit: [0] number of moves, then max_moves sources, then max_moves destinations
  const int32_t* block_table;
  int B, K, S_max, keep, sinks, max_moves, cluster, seg_keys;
  int num_blocks, block_size, max_blocks, row_chunks, ctas_per_unit;
};

// Scores in an order-preserving unsigned form: larger is better, NaN 0, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;  // -inf 0x007fffff .. +inf 0xff800000
}

// recent: positions from here on are held (64 bits: above every position when no row is held for its age)
__device__ __forceinline__ uint32_t evict_key(const EvictParams& p, size_t base, int t, long long recent) {
  const int pos = p.row_pos ? p.row_pos[base + t] : t;
  if (pos < p.sinks || pos >= recent) return 0xffffffffu;
  return score_key(p.scores[base + t]);
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t ev_smem[];
  uint32_t* hist = ev_smem;                                         // [kEvBins]
  int* wcount = reinterpret_cast<int*>(ev_smem + kEvBins);          // [4][kEvWarps]
  int* shared = wcount + 4 * kEvWarps;                              // [16] CTA totals and results
  uint32_t* keys = reinterpret_cast<uint32_t*>(shared + 16);        // [seg_keys]
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), nranks = p.cluster;
  const int unit = blockIdx.x / nranks;
  const int b = unit / p.K;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();

  int32_t* list = p.ws + (size_t)unit * (1 + 2 * (size_t)p.max_moves);
  const int len = p.seqlens[b];
  if (len <= p.keep || len > p.S_max) {  // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      list[0] = 0;
      if ((len < 0 || len > p.S_max) && unit % p.K == 0) raise_error(GQA_DEVERR_SEQLEN);
    }
    return;
  }
  const size_t base = (size_t)unit * p.S_max;
  const long long recent = p.recent_from ? (long long)p.recent_from[b] : 1ll << 32;
  const int seg = ((len + nranks - 1) / nranks + 31) / 32 * 32;
  const int t0 = min(len, rank * seg), t1 = min(len, t0 + seg);
  const int held = min(t1 - t0, p.seg_keys);
  auto key_of = [&](int i) {  // key of row t0 + i
    return i < held ? keys[i] : evict_key(p, base, t0 + i, recent);
  };
  for (int i = tid; i < held; i += kEvThreads) keys[i] = evict_key(p, base, t0 + i, recent);

  // ---- tau, the keep-th largest key, and how many rows equal to it stay
  uint32_t prefix = 0, mask = 0;
  int need = p.keep;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kBits[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int nb = 1 << kBits[pass];
    for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0u;
    __syncthreads();
    for (int i = tid; i < t1 - t0; i += kEvThreads) {
      const uint32_t k = key_of(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> kShift[pass]) & (nb - 1)], 1u);
    }
    cl.sync();
    // thread i: bins nb-1-2i and nb-2-2i (from the top), summed over the cluster
    int c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int bin = nb - 1 - (2 * tid + j);
      c[j] = 0;
      if (bin >= 0)
        for (int r = 0; r < nranks; ++r) c[j] += (int)cl.map_shared_rank(hist, r)[bin];
    }
    int incl = c[0] + c[1];  // inclusive scan over threads: keys in this thread's bins or higher
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) wcount[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += wcount[w];
    const int above = before + incl - c[0] - c[1];  // keys in higher bins than this thread's
    if (above < need && above + c[0] + c[1] >= need) {  // exactly one thread
      const bool first = above + c[0] >= need;
      shared[0] = nb - 1 - (2 * tid + (first ? 0 : 1));
      shared[1] = need - above - (first ? 0 : c[0]);
    }
    __syncthreads();
    prefix |= (uint32_t)shared[0] << kShift[pass];
    mask |= (uint32_t)(nb - 1) << kShift[pass];
    need = shared[1];
    cl.sync();  // every CTA has read this histogram
  }
  const uint32_t tau = prefix;
  const int need_eq = need;  // of the rows equal to tau, the first need_eq stay

  // ---- rows equal to tau before each warp's share of the segment
  const int wseg = ((t1 - t0 + kEvWarps - 1) / kEvWarps + 31) / 32 * 32;
  const int w0 = min(t1 - t0, warp * wseg), w1 = min(t1 - t0, w0 + wseg);
  int eq = 0;
  for (int i = w0 + lane; i < w1; i += 32) eq += key_of(i) == tau;
  eq = warp_sum(eq);
  if (lane == 0) wcount[warp] = eq;
  __syncthreads();
  if (tid == 0) {
    int s = 0;
    for (int w = 0; w < kEvWarps; ++w) s += wcount[w];
    shared[2] = s;
  }
  cl.sync();
  int eq_before = 0;
  for (int r = 0; r < rank; ++r) eq_before += cl.map_shared_rank(shared, r)[2];
  for (int w = 0; w < warp; ++w) eq_before += wcount[w];

  // ---- holes and movers, counted and then numbered
  auto sweep = [&](int holes, int movers, bool write) {
    int e = eq_before;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < w1;
      const uint32_t k = in ? key_of(i) : 0u;
      const bool is_eq = in && k == tau;
      const unsigned below = (1u << lane) - 1u;
      const unsigned em = __ballot_sync(0xffffffffu, is_eq);
      const bool stays = in && (k > tau || (is_eq && e + __popc(em & below) < need_eq));
      e += __popc(em);
      const int t = t0 + i;
      const bool hole = in && t < p.keep && !stays, mover = in && t >= p.keep && stays;
      const unsigned hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
      if (write) {
        if (mover) list[1 + movers + __popc(mm & below)] = t;
        if (hole) list[1 + p.max_moves + holes + __popc(hm & below)] = t;
      }
      holes += __popc(hm);
      movers += __popc(mm);
    }
    return make_int2(holes, movers);
  };
  const int2 mine = sweep(0, 0, false);
  if (lane == 0) {
    wcount[kEvWarps + warp] = mine.x;
    wcount[2 * kEvWarps + warp] = mine.y;
  }
  __syncthreads();
  if (tid == 0) {
    int h = 0, m = 0;
    for (int w = 0; w < kEvWarps; ++w) {
      h += wcount[kEvWarps + w];
      m += wcount[2 * kEvWarps + w];
    }
    shared[3] = h;
    shared[4] = m;
  }
  cl.sync();
  int holes = 0, movers = 0, moves = 0;
  for (int r = 0; r < nranks; ++r) {
    const int* o = cl.map_shared_rank(shared, r);
    if (r < rank) {
      holes += o[3];
      movers += o[4];
    }
    moves += o[4];
  }
  for (int w = 0; w < warp; ++w) {
    holes += wcount[kEvWarps + w];
    movers += wcount[2 * kEvWarps + w];
  }
  sweep(holes, movers, true);
  __threadfence();
  cl.sync();  // the lists are complete, and no CTA reads another's shared memory from here on

  // ---- scores and positions along with their rows, then the rows past keep
  for (int i = rank * kEvThreads + tid; i < moves; i += nranks * kEvThreads) {
    const int src = __ldcg(list + 1 + i), dst = __ldcg(list + 1 + p.max_moves + i);
    p.scores[base + dst] = p.scores[base + src];
    if (p.row_pos) p.row_pos[base + dst] = p.row_pos[base + src];
  }
  cl.sync();
  for (int t = p.keep + rank * kEvThreads + tid; t < len; t += nranks * kEvThreads) {
    p.scores[base + t] = 0.f;
    if (p.row_pos) p.row_pos[base + t] = -1;
  }
  if (rank == 0 && tid == 0) list[0] = moves;
}

constexpr int kEvMoveThreads = 256;

// Chunk index of row t of unit (b, g), or -1 (a table entry outside the pool).
__device__ __forceinline__ long long evict_row(const EvictParams& p, int b, int g, int t) {
  if (p.block_table == nullptr) return (((long long)b * p.K + g) * p.S_max + t) * p.row_chunks;
  const int blk = __ldg(p.block_table + (size_t)b * p.max_blocks + t / p.block_size);
  if ((unsigned)blk >= (unsigned)p.num_blocks) {
    raise_error(GQA_DEVERR_BLOCK);
    return -1;
  }
  return (((long long)blk * p.K + g) * p.block_size + t % p.block_size) * p.row_chunks;
}

// ctas_per_unit CTAs per unit; row_chunks 16-byte lanes per row and tensor.
// The first CTA of a sequence's first unit also writes its new length: every
// unit's list is complete when this kernel starts, and nothing here reads a
// length but that thread.
__global__ void __launch_bounds__(kEvMoveThreads) evict_move_kernel(const EvictParams p) {
  const int unit = blockIdx.x / p.ctas_per_unit, part = blockIdx.x % p.ctas_per_unit;
  const int b = unit / p.K, g = unit % p.K;
  grid_dep_wait();
  grid_dep_launch();
  if (part == 0 && g == 0 && threadIdx.x == 0) {
    const int len = p.seqlens[b];
    if (len > p.keep && len <= p.S_max) p.seqlens[b] = p.keep;
  }
  const int32_t* list = p.ws + (size_t)unit * (1 + 2 * (size_t)p.max_moves);
  const int moves = __ldcg(list);
  const int lanes = 2 * p.row_chunks;  // K's chunks, then V's
  const int per_cta = kEvMoveThreads / lanes;
  const int c = threadIdx.x % lanes;
  const bool is_v = c >= p.row_chunks;
  const int ch = is_v ? c - p.row_chunks : c;
  uint4* cache = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache);
  constexpr int U = 4;  // rows in flight per lane group
  for (int i0 = part * per_cta * U + threadIdx.x / lanes; i0 < moves; i0 += p.ctas_per_unit * per_cta * U) {
    long long src[U], dst[U];
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * per_cta;
      src[u] = dst[u] = -1;
      if (i < moves) {
        src[u] = evict_row(p, b, g, __ldcg(list + 1 + i));
        dst[u] = evict_row(p, b, g, __ldcg(list + 1 + p.max_moves + i));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0 && dst[u] >= 0) w[u] = cache[src[u] + ch];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0 && dst[u] >= 0) cache[dst[u] + ch] = w[u];
  }
}

}  // namespace gqa
