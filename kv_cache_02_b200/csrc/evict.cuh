// gqa_kv_evict: which rows stay, and the moves that close the cache up.
//
// A row's rank is a 32-bit key, the larger the better: held rows all ones,
// others their score mapped to an order-preserving integer (NaN 0). The rows
// that stay are the `keep` largest keys, the lower row first among equal ones:
// those above the keep-th largest key tau, and the first need_eq rows equal to
// it. Then the holes (rows below keep that go) and the movers (rows from keep
// on that stay) are numbered in order of their rows: mover i goes to hole i.
//
//   evict_cta_kernel     bounded caches (at most kEvCtaRows): a CTA per (b, g),
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
//     The movers' scores and positions go to the workspace with their numbers,
//     so that the rows past keep can be cleared at once, by the threads that
//     own them.
//   evict_move_kernel    all CTAs of the GPU, a group of lanes per row: sources
//     lie at or above keep and destinations below it, so no order is needed.
//
// Bytes: 8 per row read (score, position), and the moved rows twice. Measured:
// 64 heads cut from about 2080 rows to 2048, one launch: 10 us; 8 heads from
// 131072 rows to 8192: select 27 us, move 17 us (62 MB in rows of 256 bytes).
// What is left of the select is one cluster barrier and two reads of other
// CTAs' histograms a pass (3 us), and 16 keys a thread looked at five times.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "decode.cuh"

namespace gqa {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
static_assert(kEvWarps == 32, "a lane per warp joins the warps' counts");
constexpr int kEvCtaRows = 16384;    // evict_cta_kernel: up to 16 rows a thread
// Moves that the CTA makes itself rather than a kernel of their own: 64 heads of 2080 rows to 2048 (256 at most) 10.4
// us against 11.2, 2304 to 512 (512 at most) 15.8 against 18.1; at 2048 at most (2560 rows to 2048) 64 heads still
// gain (15.9 against 17.9), but 8 heads, which leave most SMs idle, lose (14.0 against 10.4).
constexpr int kEvFusedMoves = 512;
constexpr int kEvBins = 2048;
constexpr int kEvCopies = 4;         // histograms of a CTA: fewer warps meet in a bin
constexpr int kEvCluster = 8;
constexpr int kEvFine = 32;          // bins of a coarse bin: a cluster sums the coarse ones, then one's fine ones
constexpr int kEvStaticBytes = ((kEvCopies + 2) * kEvBins + 2 * (kEvBins / kEvFine) + 4 * kEvWarps + 16) * 4;
// keys of a segment kept in shared memory; rows past these (caches of more than 8 x 40960 rows) are read again
constexpr int kEvMaxSegKeys = 40960;

struct EvictParams {
  void *k_cache, *v_cache;
  float* scores;
  int32_t* row_pos;  // or null
  int32_t* seqlens;
  const int32_t* recent_from;  // or null
  int32_t* ws;                 // per unit: the number of moves, then max_moves each of sources, destinations,
                               // scores (float bits) and positions
  unsigned long long* done;    // fused moves: [B] tagged counters of the heads that are done
  unsigned long long tag;
  const int32_t* block_table;
  int B, K, S_max, keep, sinks, max_moves, seg_keys;
  int quads;  // scores and positions may be read four at a time
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
  const int blk = __ldcg(p.block_table + (size_t)b * p.max_blocks + t / p.block_size);
  if ((unsigned)blk >= (unsigned)p.num_blocks) {
    raise_error(GQA_DEVERR_BLOCK);
    return -1;
  }
  return (((long long)blk * p.K + g) * p.block_size + t % p.block_size) * p.row_chunks;
}

// Rows src(i) -> dst(i), i = first, first + step, ... below n, of the lane
// group's 16-byte chunk; kEvFlight rows in flight (8 heads of 131072 rows to
// 8192: 37.7 us a call, in pages of 16 46.3, in float32 51.7; two rows 38.5,
// 47.9 and 56.4; eight 45.9, 63.2 and 70.2. 64 heads of 16384 rows to 8192: 125
// us, two rows 99, eight 155).
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

// Mover i of the unit: its row, score and position to the workspace
__device__ __forceinline__ void evict_save(const EvictParams& p, int32_t* list, int i, int t, float score, int pos) {
  list[1 + i] = t;
  list[1 + 2 * (size_t)p.max_moves + i] = __float_as_int(score);
  if (p.row_pos) list[1 + 3 * (size_t)p.max_moves + i] = pos;
}

__device__ __forceinline__ void evict_clear(const EvictParams& p, size_t at) {
  p.scores[at] = 0.f;
  if (p.row_pos) p.row_pos[at] = -1;
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
  int32_t* list = p.ws + (size_t)unit * (1 + 4 * (size_t)p.max_moves);
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
  int32_t* to = kFused ? moved + kEvFusedMoves : list + 1 + p.max_moves;
  float score[J];
  int pos[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {  // the separate moves' scores and positions, asked for together
    const int t = row0 + j * 32;
    const bool ask = !kFused && t >= p.keep && t < end;
    score[j] = ask ? p.scores[base + t] : 0.f;
    pos[j] = ask && p.row_pos ? p.row_pos[base + t] : 0;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int t = row0 + j * 32;
    const bool s = stay >> j & 1;
    const bool hole = t < min(end, p.keep) && !s, mover = t >= p.keep && s;
    const unsigned below = (1u << lane) - 1u;
    const unsigned hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    if (mover) {
      const int i = movers + __popc(mb & below);
      if (kFused)
        moved[i] = t;
      else
        evict_save(p, list, i, t, score[j], pos[j]);
    }
    if (hole) to[holes + __popc(hb & below)] = t;
    if (!kFused && t >= p.keep && t < end) evict_clear(p, base + t);
    holes += __popc(hb);
    movers += __popc(mb);
  }
  if (!kFused) {
    if (tid == 0) list[0] = moves;
    return;
  }
  __syncthreads();

  // ---- rows, scores and positions, then the rows past keep
  for (int i = tid; i < moves; i += kEvThreads) {
    p.scores[base + to[i]] = p.scores[base + moved[i]];
    if (p.row_pos) p.row_pos[base + to[i]] = p.row_pos[base + moved[i]];
  }
  {
    const int lanes = 2 * p.row_chunks;  // K's chunks, then V's
    evict_move_rows(p, b, g, tid % lanes, tid / lanes, kEvThreads / lanes, moves, [&](int i) { return moved[i]; },
                    [&](int i) { return moved[kEvFusedMoves + i]; });
  }
  __syncthreads();
  for (int t = p.keep + tid; t < len; t += kEvThreads) evict_clear(p, base + t);
  if (tid == 0) {
    // the length: written once every head of the sequence has read it
    __threadfence();
    if (take_ticket(p.done + b, p.tag) == p.K) {
      __threadfence();
      p.seqlens[b] = p.keep;
      *reinterpret_cast<volatile unsigned long long*>(p.done + b) = 0ull;  // a replay repeats the tag
    }
  }
}

__global__ void __cluster_dims__(kEvCluster, 1, 1) __launch_bounds__(kEvThreads)
    evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t ev_smem[];
  uint32_t* hist = ev_smem;                                              // [kEvCopies][kEvBins]
  uint32_t* sums = hist + kEvCopies * kEvBins;                           // [pass parity][kEvBins] the copies' sums
  uint32_t* coarse = sums + 2 * kEvBins;                                 // [pass parity][kEvBins / kEvFine]
  int* wcount = reinterpret_cast<int*>(coarse + 2 * (kEvBins / kEvFine));  // [4][kEvWarps]
  int* shared = wcount + 4 * kEvWarps;                                   // [16] CTA totals and results
  uint32_t* keys = reinterpret_cast<uint32_t*>(shared + 16);             // [seg_keys]
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int unit = blockIdx.x / kEvCluster;
  const int b = unit / p.K;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();

  int32_t* list = p.ws + (size_t)unit * (1 + 4 * (size_t)p.max_moves);
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
  uint32_t* mine = hist + (warp % kEvCopies) * kEvBins;
  for (int i = tid; i < kEvCopies * kEvBins; i += kEvThreads) hist[i] = 0u;
  __syncthreads();

  // ---- tau, the keep-th largest key, and how many rows equal to it stay
  uint32_t prefix = 0, mask = 0;
  int need = p.keep;
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kBits[3] = {11, 11, 10};
  // the keys, and the first histogram with them
  const int quads = p.quads ? held / 4 : 0;
#pragma unroll 4
  for (int i = tid; i < quads; i += kEvThreads) {
    const float4 sc = *reinterpret_cast<const float4*>(p.scores + base + t0 + 4 * i);
    int4 at = make_int4(t0 + 4 * i, t0 + 4 * i + 1, t0 + 4 * i + 2, t0 + 4 * i + 3);
    if (p.row_pos) at = *reinterpret_cast<const int4*>(p.row_pos + base + t0 + 4 * i);
    auto key = [&](float v, int pos) { return pos < p.sinks || pos >= recent ? 0xffffffffu : score_key(v); };
    const uint4 k = make_uint4(key(sc.x, at.x), key(sc.y, at.y), key(sc.z, at.z), key(sc.w, at.w));
    reinterpret_cast<uint4*>(keys)[i] = k;
    atomicAdd(&mine[k.x >> kShift[0]], 1u);
    atomicAdd(&mine[k.y >> kShift[0]], 1u);
    atomicAdd(&mine[k.z >> kShift[0]], 1u);
    atomicAdd(&mine[k.w >> kShift[0]], 1u);
  }
  for (int i = 4 * quads + tid; i < t1 - t0; i += kEvThreads) {
    const uint32_t k = evict_key(p, base, t0 + i, recent);
    if (i < held) keys[i] = k;
    atomicAdd(&mine[k >> kShift[0]], 1u);
  }

  bool exact = false;  // as many keys with this prefix or above as rows stay
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    if (exact) break;
    const int nb = 1 << kBits[pass];
    uint32_t* sum = sums + (pass & 1) * kEvBins;
    if (pass > 0) {
      for (int i = tid; i < kEvCopies * kEvBins; i += kEvThreads) hist[i] = 0u;
      __syncthreads();
      auto add = [&](uint32_t k) {
        if ((k & mask) == prefix) atomicAdd(&mine[(k >> kShift[pass]) & (nb - 1)], 1u);
      };
#pragma unroll 4
      for (int i = tid; i < held / 4; i += kEvThreads) {
        const uint4 k = reinterpret_cast<const uint4*>(keys)[i];
        add(k.x), add(k.y), add(k.z), add(k.w);
      }
      for (int i = held / 4 * 4 + tid; i < t1 - t0; i += kEvThreads) add(key_of(i));
    }
    __syncthreads();
    // bins 2 tid and 2 tid + 1: the copies' sums, and 16 lanes' coarse bin
    if (tid < nb / 2) {
      uint2 c = make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < kEvCopies; ++i) {
        const uint2 v = reinterpret_cast<const uint2*>(hist + i * kEvBins)[tid];
        c.x += v.x, c.y += v.y;
      }
      reinterpret_cast<uint2*>(sum)[tid] = c;
      uint32_t all = c.x + c.y;
#pragma unroll
      for (int off = kEvFine / 4; off > 0; off >>= 1) all += __shfl_xor_sync(0xffffffffu, all, off);
      if ((lane & 15) == 0) coarse[(pass & 1) * (kEvBins / kEvFine) + tid / 16] = all;
    }
    // (a sum's second use comes after the next pass's: every CTA has read its first by then)
    cl.sync();
    if (warp == 0) {
      // the bin, counted from the top, that the need-th key lies in: among the coarse ones (two a lane), then among
      // its fine ones. c0: the higher of the lane's bins, c1: the lower
      auto find = [&](int c0, int c1, int want, int& at, int& above, int& count) {
        int incl = c0 + c1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += o;
        }
        const int before = incl - c0 - c1;
        const unsigned hit = __ballot_sync(0xffffffffu, before < want && incl >= want);  // one lane
        const int who = __ffs(hit) - 1;
        const bool low = before + c0 < want;
        at = __shfl_sync(0xffffffffu, 2 * lane + (low ? 1 : 0), who);
        above = __shfl_sync(0xffffffffu, low ? before + c0 : before, who);
        count = __shfl_sync(0xffffffffu, low ? c1 : c0, who);
      };
      const int nc = nb / kEvFine;  // 64 or 32
      int c0 = 0, c1 = 0;
#pragma unroll
      for (int r = 0; r < kEvCluster; ++r) {
        const uint32_t* v = cl.map_shared_rank(coarse, r) + (pass & 1) * (kEvBins / kEvFine);
        if (2 * lane < nc) {
          c0 += (int)v[nc - 1 - 2 * lane];
          c1 += (int)v[nc - 2 - 2 * lane];
        }
      }
      int group, above, count, fine, fine_above;
      find(c0, c1, need, group, above, count);
      group = nc - 1 - group;
      c0 = 0;
#pragma unroll
      for (int r = 0; r < kEvCluster; ++r)
        c0 += (int)cl.map_shared_rank(sum, r)[group * kEvFine + kEvFine - 1 - lane];
      find(c0, 0, need - above, fine, fine_above, count);
      if (lane == 0) {
        shared[0] = group * kEvFine + kEvFine - 1 - fine / 2;
        shared[1] = need - above - fine_above;
        shared[5] = shared[1] == count;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)shared[0] << kShift[pass];
    mask |= (uint32_t)(nb - 1) << kShift[pass];
    need = shared[1];
    exact = shared[5] != 0 && prefix != 0;
    __syncthreads();  // before they are written again
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
  // kBatch x 32 rows at a time: the rows' scores and positions, if they are to be written, are all asked for first
  constexpr int kBatch = 4;
  auto sweep = [&](int holes, int movers, auto write) {
    int e = eq_before;
    for (int i0 = w0; i0 < w1; i0 += 32 * kBatch) {
      float score[kBatch];
      int pos[kBatch];
      if constexpr (write.value) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = i0 + 32 * u + lane, t = t0 + i;
          const bool ask = i < w1 && t >= p.keep && key_of(i) >= tau;
          score[u] = ask ? p.scores[base + t] : 0.f;
          pos[u] = ask && p.row_pos ? p.row_pos[base + t] : 0;
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + 32 * u + lane;
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
        if constexpr (write.value) {
          if (mover) evict_save(p, list, movers + __popc(mm & below), t, score[u], pos[u]);
          if (hole) list[1 + p.max_moves + holes + __popc(hm & below)] = t;
        }
        holes += __popc(hm);
        movers += __popc(mm);
      }
    }
    return make_int2(holes, movers);
  };
  int2 found;
  if (need_eq == 0 && held == t1 - t0) {  // no ties, all keys at hand: no order is needed to count
    int below = 0, beyond = 0;
    const int first = p.keep - t0;  // row t0 + i is below keep for i < first
#pragma unroll 2
    for (int i = w0 + 4 * lane; i < w1; i += 128) {
      const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
      const uint32_t kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < w1) {
          below += kk[j] <= tau && i + j < first;
          beyond += kk[j] > tau && i + j >= first;
        }
    }
    found = make_int2(warp_sum(below), warp_sum(beyond));
  } else {
    found = sweep(0, 0, std::false_type());
  }
  if (lane == 0) {
    wcount[kEvWarps + warp] = found.x;
    wcount[2 * kEvWarps + warp] = found.y;
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
  cl.barrier_arrive();  // done with the other CTAs' shared memory
  sweep(holes, movers, std::true_type());
  if (rank == 0 && tid == 0) list[0] = moves;
  __syncthreads();  // the movers' scores have been read
  const int clear0 = max(t0, p.keep);
  const int quad0 = p.quads ? (clear0 + 3) / 4 : 0, quad1 = p.quads ? t1 / 4 : 0;  // of four rows each
  for (int i = quad0 + tid; i < quad1; i += kEvThreads) {
    reinterpret_cast<float4*>(p.scores + base)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.row_pos) reinterpret_cast<int4*>(p.row_pos + base)[i] = make_int4(-1, -1, -1, -1);
  }
  const bool any = quad0 < quad1;
  for (int t = clear0 + tid; t < (any ? min(t1, 4 * quad0) : t1); t += kEvThreads) evict_clear(p, base + t);
  if (any)
    for (int t = 4 * quad1 + tid; t < t1; t += kEvThreads) evict_clear(p, base + t);
  cl.barrier_wait();
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
  const int32_t* list = p.ws + (size_t)unit * (1 + 4 * (size_t)p.max_moves);
  const int moves = __ldcg(list);
  const size_t base = (size_t)unit * p.S_max, mm = p.max_moves;
  for (int i = part * kEvMoveThreads + threadIdx.x; i < moves; i += p.ctas_per_unit * kEvMoveThreads) {
    const int to = __ldcg(list + 1 + mm + i);
    p.scores[base + to] = __int_as_float(__ldcg(list + 1 + 2 * mm + i));
    if (p.row_pos) p.row_pos[base + to] = __ldcg(list + 1 + 3 * mm + i);
  }
  const int lanes = 2 * p.row_chunks, per_cta = kEvMoveThreads / lanes;  // K's chunks, then V's
  evict_move_rows(p, b, g, threadIdx.x % lanes, part * per_cta + threadIdx.x / lanes, p.ctas_per_unit * per_cta, moves,
                  [&](int i) { return __ldcg(list + 1 + i); }, [&](int i) { return __ldcg(list + 1 + p.max_moves + i); });
}

}  // namespace gqa
