// gqa_kv_evict: which rows stay, and the moves that close the cache up.
//
// A row's rank is a 32-bit key, the larger the better: held rows all ones,
// others their score mapped to an order-preserving integer (NaN 0). The rows
// that stay are the `keep` largest keys, the lower row first among equal ones:
// those above the keep-th largest key tau, and the first need_eq rows equal to
// it. Then the holes (rows below keep that go) and the movers (rows from keep
// on that stay) are numbered in order of their rows: mover i goes to hole i.
//
//   evict_cta_kernel     bounded caches (kEvCtaRows rows): a CTA per (b, g),
//     keys in registers. tau two bits a round, the counts of three candidates
//     exchanged behind one barrier; as soon as one of them counts keep rows,
//     that is the answer (random scores: about 11 of 16 rounds). With few
//     moves (kEvFusedMoves at most) the CTA makes them itself, and the last of
//     a sequence's heads writes its length: one launch. A step's latency is
//     what bounds it.
//   evict_select_kernel  longer ones: a cluster of CTAs per (b, g), each with a
//     contiguous segment of the rows, whose keys it reads once and keeps in
//     shared memory (S_max 131072: 8 CTAs of 64 KB). tau by a radix select, 11
//     + 11 + 10 bits, the histograms summed over the cluster through
//     distributed shared memory.
//   evict_move_kernel    all CTAs of the GPU, a group of lanes per row: sources
//     lie at or above keep and destinations below it, so no order is needed.
//
// Bytes: 8 per row read (score, position), and the moved rows twice.
#pragma once

#include <cooperative_groups.h>

#include "common.cuh"
#include "decode.cuh"

namespace gqa {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
static_assert(kEvWarps == 32, "a lane per warp joins the warps' counts");
constexpr int kEvCtaRows = 8192;     // evict_cta_kernel: up to 8 rows a thread
constexpr int kEvFusedMoves = 512;
constexpr int kEvBins = 2048;
constexpr int kEvCopies = 4;         // histograms of a CTA: fewer warps meet in a bin
constexpr int kEvCluster = 8;
constexpr int kEvStaticBytes = (kEvCopies * kEvBins + 4 * kEvWarps + 16) * 4;
// keys of a segment kept in shared memory; rows past these (caches of more than 8 x 40960 rows) are read again
constexpr int kEvMaxSegKeys = 40960;

struct EvictParams {
  void *k_cache, *v_cache;
  float* scores;
  int32_t* row_pos;  // or null
  int32_t* seqlens;
  const int32_t* recent_from;  // or null
  int32_t* ws;                 // per unit: [0] number of moves, then max_moves sources, then max_moves destinations
  unsigned long long* done;    // fused moves: [B] tagged counters of the heads that are done
  unsigned long long tag;
  const int32_t* block_table;
  int B, K, S_max, keep, sinks, max_moves, seg_keys;
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
  const uint32_t key = score_key(p.scores[base + t]);  // asked for along with the position
  return pos < p.sinks || pos >= recent ? 0xffffffffu : key;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

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

// Rows src(i) -> dst(i), i = first, first + step, ... below n, of the lane
// group's 16-byte chunk; kEvFlight rows in flight.
constexpr int kEvFlight = 4;
template <typename Src, typename Dst>
__device__ __forceinline__ void evict_move_rows(const EvictParams& p, int b, int g, int lane, int first, int step, int n,
                                                Src src, Dst dst) {
  const bool is_v = lane >= p.row_chunks;
  uint4* cache = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache) + (is_v ? lane - p.row_chunks : lane);
  for (int i0 = first; i0 < n; i0 += kEvFlight * step) {
    long long from[kEvFlight], to[kEvFlight];
    uint4 w[kEvFlight];
#pragma unroll
    for (int u = 0; u < kEvFlight; ++u) {
      const int i = i0 + u * step;
      from[u] = to[u] = -1;
      if (i < n) {
        from[u] = evict_row(p, b, g, src(i));
        to[u] = evict_row(p, b, g, dst(i));
      }
    }
#pragma unroll
    for (int u = 0; u < kEvFlight; ++u)
      if (from[u] >= 0 && to[u] >= 0) w[u] = cache[from[u]];
#pragma unroll
    for (int u = 0; u < kEvFlight; ++u)
      if (from[u] >= 0 && to[u] >= 0) cache[to[u]] = w[u];
  }
}

// Sum of v over the lanes below n, and over all
__device__ __forceinline__ int2 below_and_all(int v, int n) {
  const int lane = threadIdx.x & 31;
  return make_int2(warp_sum(lane < n ? v : 0), warp_sum(v));
}

// J: rows of a thread, at most. Warp w holds rows w * seg .., 32 at a time.
template <int J, bool kFused>
__global__ void __launch_bounds__(kEvThreads) evict_cta_kernel(const EvictParams p) {
  __shared__ uint2 counts[2][kEvWarps];
  __shared__ int held_eq[kEvWarps];
  __shared__ int2 hm[kEvWarps];
  __shared__ int moved[kFused ? 2 * kEvFusedMoves : 1];
  const int unit = blockIdx.x;
  const int b = unit / p.K, g = unit % p.K;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  int32_t* list = p.ws + (size_t)unit * (1 + 2 * (size_t)p.max_moves);
  const int len = p.seqlens[b];
  const long long recent = p.recent_from ? (long long)p.recent_from[b] : 1ll << 32;
  if (len <= p.keep || len > p.S_max) {
    if (tid == 0) {
      if (!kFused) list[0] = 0;
      if ((len < 0 || len > p.S_max) && g == 0) raise_error(GQA_DEVERR_SEQLEN);
    }
    return;
  }
  const size_t base = (size_t)unit * p.S_max;
  const int seg = (len + kEvThreads - 1) / kEvThreads * 32;
  const int row0 = warp * seg + lane, end = min(len, (warp + 1) * seg);
  uint32_t key[J];
#pragma unroll
  for (int j = 0; j < J; ++j) key[j] = row0 + j * 32 < end ? evict_key(p, base, row0 + j * 32, recent) : 0u;

  // ---- tau: the largest key that at least keep keys reach
  uint32_t tau = 0;
  int reach = len;  // keys >= tau
#pragma unroll 1
  for (int s = 30, round = 0; s >= 0 && reach != p.keep; s -= 2, ++round) {
    const uint32_t c1 = tau | (1u << s), c2 = tau | (2u << s), c3 = tau | (3u << s);
    uint32_t n12 = 0, n3 = 0;  // a row past the end has key 0 and reaches none
#pragma unroll
    for (int j = 0; j < J; ++j) {
      n12 += (key[j] >= c1 ? 1u : 0u) + (key[j] >= c2 ? 0x10000u : 0u);
      n3 += key[j] >= c3 ? 1u : 0u;
    }
    n12 = __reduce_add_sync(0xffffffffu, n12);
    n3 = __reduce_add_sync(0xffffffffu, n3);
    if (lane == 0) counts[round & 1][warp] = make_uint2(n12, n3);
    __syncthreads();
    const uint2 c = counts[round & 1][lane];
    n12 = __reduce_add_sync(0xffffffffu, c.x);
    n3 = __reduce_add_sync(0xffffffffu, c.y);
    const int k1 = (int)(n12 & 0xffffu), k2 = (int)(n12 >> 16), k3 = (int)n3;
    if (k3 >= p.keep)
      tau = c3, reach = k3;
    else if (k2 >= p.keep)
      tau = c2, reach = k2;
    else if (k1 >= p.keep)
      tau = c1, reach = k1;
  }
  // of the rows equal to tau all stay (reach == keep), or the first need_eq
  unsigned stay = 0;  // bit j: row j of the thread
  if (reach == p.keep) {
#pragma unroll
    for (int j = 0; j < J; ++j) stay |= (row0 + j * 32 < end && key[j] >= tau ? 1u : 0u) << j;
  } else {
    int eq = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) eq += row0 + j * 32 < end && key[j] == tau;
    eq = warp_sum(eq);
    if (lane == 0) held_eq[warp] = eq;
    __syncthreads();
    const int2 e = below_and_all(held_eq[lane], warp);
    const int need_eq = p.keep - (reach - e.y);
    int rank = e.x;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool in = row0 + j * 32 < end, is_eq = in && key[j] == tau;
      const unsigned m = __ballot_sync(0xffffffffu, is_eq);
      const bool s = in && (key[j] > tau || (is_eq && rank + __popc(m & ((1u << lane) - 1u)) < need_eq));
      stay |= (s ? 1u : 0u) << j;
      rank += __popc(m);
    }
  }

  // ---- holes and movers, counted and then numbered
  int holes = 0, movers = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int t = row0 + j * 32;
    const bool s = stay >> j & 1;
    holes += t < min(end, p.keep) && !s;
    movers += t >= p.keep && s;
  }
  holes = warp_sum(holes);
  movers = warp_sum(movers);
  if (lane == 0) hm[warp] = make_int2(holes, movers);
  __syncthreads();
  const int2 h = below_and_all(hm[lane].x, warp), m = below_and_all(hm[lane].y, warp);
  const int moves = m.y;
  holes = h.x;
  movers = m.x;
  int32_t* from = kFused ? moved : list + 1;
  int32_t* to = kFused ? moved + kEvFusedMoves : list + 1 + p.max_moves;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int t = row0 + j * 32;
    const bool s = stay >> j & 1;
    const bool hole = t < min(end, p.keep) && !s, mover = t >= p.keep && s;
    const unsigned below = (1u << lane) - 1u;
    const unsigned hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    if (mover) from[movers + __popc(mb & below)] = t;
    if (hole) to[holes + __popc(hb & below)] = t;
    holes += __popc(hb);
    movers += __popc(mb);
  }
  __syncthreads();  // (the workspace's lists too: written and read by this CTA)

  // ---- scores and positions along with their rows, then the rows past keep
  for (int i = tid; i < moves; i += kEvThreads) {
    p.scores[base + to[i]] = p.scores[base + from[i]];
    if (p.row_pos) p.row_pos[base + to[i]] = p.row_pos[base + from[i]];
  }
  if (kFused) {
    const int lanes = 2 * p.row_chunks;  // K's chunks, then V's
    evict_move_rows(p, b, g, tid % lanes, tid / lanes, kEvThreads / lanes, moves, [&](int i) { return moved[i]; },
                    [&](int i) { return moved[kEvFusedMoves + i]; });
  }
  __syncthreads();
  for (int t = p.keep + tid; t < len; t += kEvThreads) {
    p.scores[base + t] = 0.f;
    if (p.row_pos) p.row_pos[base + t] = -1;
  }
  if (tid == 0) {
    if (!kFused) {
      list[0] = moves;
    } else {
      // the length: written once every head of the sequence has read it
      __threadfence();
      if (take_ticket(p.done + b, p.tag) == p.K) {
        __threadfence();
        p.seqlens[b] = p.keep;
        *reinterpret_cast<volatile unsigned long long*>(p.done + b) = 0ull;  // a replay repeats the tag
      }
    }
  }
}

__global__ void __cluster_dims__(kEvCluster, 1, 1) __launch_bounds__(kEvThreads)
    evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t ev_smem[];
  uint32_t* hist = ev_smem;                                              // [kEvCopies][kEvBins]
  int* wcount = reinterpret_cast<int*>(ev_smem + kEvCopies * kEvBins);   // [4][kEvWarps]
  int* shared = wcount + 4 * kEvWarps;                                   // [16] CTA totals and results
  uint32_t* keys = reinterpret_cast<uint32_t*>(shared + 16);             // [seg_keys]
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int unit = blockIdx.x / kEvCluster;
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
  const int seg = ((len + kEvCluster - 1) / kEvCluster + 31) / 32 * 32;
  const int t0 = min(len, rank * seg), t1 = min(len, t0 + seg);
  const int held = min(t1 - t0, p.seg_keys);
  auto key_of = [&](int i) {  // key of row t0 + i
    return i < held ? keys[i] : evict_key(p, base, t0 + i, recent);
  };
#pragma unroll 4
  for (int i = tid; i < held; i += kEvThreads) keys[i] = evict_key(p, base, t0 + i, recent);
  __syncthreads();

  // ---- tau, the keep-th largest key, and how many rows equal to it stay
  uint32_t prefix = 0, mask = 0;
  int need = p.keep;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kBits[3] = {11, 11, 10};
  bool exact = false;  // as many keys with this prefix or above as rows stay
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    if (exact) break;
    const int nb = 1 << kBits[pass];
    for (int i = tid; i < kEvCopies * kEvBins; i += kEvThreads) hist[i] = 0u;
    __syncthreads();
    uint32_t* mine = hist + (warp % kEvCopies) * kEvBins;
#pragma unroll 4
    for (int i = tid; i < t1 - t0; i += kEvThreads) {
      const uint32_t k = key_of(i);
      if ((k & mask) == prefix) atomicAdd(&mine[(k >> kShift[pass]) & (nb - 1)], 1u);
    }
    __syncthreads();
    // bins 2 x and 2 x + 1, x counted from the top by thread: first over the copies, then over the cluster
    const int x = nb / 2 - 1 - tid;
    if (x >= 0) {
      uint2 c = make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < kEvCopies; ++i) {
        const uint2 v = reinterpret_cast<const uint2*>(hist + i * kEvBins)[x];
        c.x += v.x, c.y += v.y;
      }
      reinterpret_cast<uint2*>(hist)[x] = c;
    }
    cl.sync();
    int c[2] = {0, 0};  // bin 2 x + 1, bin 2 x
    if (x >= 0) {
#pragma unroll
      for (int r = 0; r < kEvCluster; ++r) {
        const uint2 v = reinterpret_cast<const uint2*>(cl.map_shared_rank(hist, r))[x];
        c[0] += (int)v.y, c[1] += (int)v.x;
      }
    }
    int incl = c[0] + c[1];  // inclusive scan over threads: keys in this thread's bins or higher
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) wcount[warp] = incl;
    __syncthreads();
    const int above = below_and_all(wcount[lane], warp).x + incl - c[0] - c[1];  // keys in higher bins than this thread's
    if (above < need && above + c[0] + c[1] >= need) {  // exactly one thread
      const bool first = above + c[0] >= need;
      shared[0] = 2 * x + (first ? 1 : 0);
      shared[1] = need - above - (first ? 0 : c[0]);
      shared[5] = shared[1] == c[first ? 0 : 1];
    }
    __syncthreads();
    prefix |= (uint32_t)shared[0] << kShift[pass];
    mask |= (uint32_t)(nb - 1) << kShift[pass];
    need = shared[1];
    exact = shared[5] != 0 && prefix != 0;
    cl.sync();  // every CTA has read this histogram
  }
  // the rows above tau stay, and of those equal to it the first need_eq
  const uint32_t tau = exact ? prefix - 1 : prefix;
  const int need_eq = exact ? 0 : need;

  // ---- rows equal to tau before each warp's share of the segment
  const int wseg = ((t1 - t0 + kEvWarps - 1) / kEvWarps + 31) / 32 * 32;
  const int w0 = min(t1 - t0, warp * wseg), w1 = min(t1 - t0, w0 + wseg);
  int eq_before = 0;
  if (need_eq > 0) {  // the same in every CTA
    int eq = 0;
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) eq += key_of(i) == tau;
    eq = warp_sum(eq);
    if (lane == 0) wcount[warp] = eq;
    __syncthreads();
    const int2 eqs = below_and_all(wcount[lane], warp);
    if (tid == 0) shared[2] = eqs.y;
    cl.sync();
    // a lane per CTA of the cluster
    eq_before = eqs.x + warp_sum(lane < rank ? cl.map_shared_rank(shared, min(lane, kEvCluster - 1))[2] : 0);
  }

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
  const int2 hw = below_and_all(wcount[kEvWarps + lane], warp), mw = below_and_all(wcount[2 * kEvWarps + lane], warp);
  if (tid == 0) {
    shared[3] = hw.y;
    shared[4] = mw.y;
  }
  cl.sync();
  const int* other = cl.map_shared_rank(shared, min(lane, kEvCluster - 1));
  const int oh = lane < kEvCluster ? other[3] : 0, om = lane < kEvCluster ? other[4] : 0;
  const int holes = hw.x + warp_sum(lane < rank ? oh : 0), movers = mw.x + warp_sum(lane < rank ? om : 0);
  const int moves = warp_sum(om);
  sweep(holes, movers, true);
  __threadfence();
  cl.sync();  // the lists are complete, and no CTA reads another's shared memory from here on

  // ---- scores and positions along with their rows, then the rows past keep
  for (int i = rank * kEvThreads + tid; i < moves; i += kEvCluster * kEvThreads) {
    const int src = __ldcg(list + 1 + i), dst = __ldcg(list + 1 + p.max_moves + i);
    p.scores[base + dst] = p.scores[base + src];
    if (p.row_pos) p.row_pos[base + dst] = p.row_pos[base + src];
  }
  cl.sync();
  for (int t = p.keep + rank * kEvThreads + tid; t < len; t += kEvCluster * kEvThreads) {
    p.scores[base + t] = 0.f;
    if (p.row_pos) p.row_pos[base + t] = -1;
  }
  if (rank == 0 && tid == 0) list[0] = moves;
}

constexpr int kEvMoveThreads = 256;

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
  const int lanes = 2 * p.row_chunks, per_cta = kEvMoveThreads / lanes;  // K's chunks, then V's
  evict_move_rows(p, b, g, threadIdx.x % lanes, part * per_cta + threadIdx.x / lanes, p.ctas_per_unit * per_cta, moves,
                  [&](int i) { return __ldcg(list + 1 + i); }, [&](int i) { return __ldcg(list + 1 + p.max_moves + i); });
}

}  // namespace gqa
