// gqa_prompt_scores: how much attention the last T queries of each sequence
// pay to each cached key, on the tensor cores (tcgen05 + TMEM + TMA).
//
//   scores[b, g, t] += sum over query rows r = (i, h in group g) of
//                      2^(x[r, t] - lse[r]),   x = scale * log2(e) * q_r . k_t
//   lse[r] = log2 sum_{t <= pos_r} 2^x[r, t],  pos_r = len_b - T + i
//
// A key's score sums over rows, a row's lse over keys, so x is computed twice,
// each time with the owner of the sum in the MMA's M dimension, where one
// thread holds it (TMEM lane = thread) and no sum crosses threads:
//   kRows  x   = Q K^T: a thread owns a query row: reference score and sum
//   kKeys  x^T = K Q^T: a thread owns a key: sum of the rows' weights, each
//          row's lse read from shared memory
// The rows of a group are taken together, r = i * G + h: a 128-row tile is
// 128 / G tokens of the G heads (fewer rows when G does not divide 128; the
// rest of the tile is zero).
//
// A work item is two stationary 128-row tiles (of Q, or of K) and the tiles of
// the other operand that they need (causal bounds drop tiles without work);
// persistent CTAs, one per SM, take items from a tagged counter, heaviest
// first. Items are split over the streamed tiles while there are too few for
// the GPU; the parts are joined in a fixed order. 18 warps:
//   warps 8 t + 4 h + q  (t, h in {0, 1}, q = 0..3): stationary tile t, columns
//            64 h .. 64 h + 63 of each streamed tile, TMEM lanes 32 q ..; the
//            two halves of a row are joined at the item's end
//   warp 16  TMEM allocation; issues the MMAs (M = N = 128, two S buffers per t)
//   warp 17  takes the items, loads their tiles: two slots of stationary tiles
//            (the next item's land while this one runs) and a ring of streams
//
// Bound: issue slots and exponentials. A pair takes one exponential per kernel,
// 16 per clock and SM in the special-function unit: 1024 clocks for a 128 x 128
// tile (512 for its MMA). kPsPoly of 16 column pairs go to the FMA pipe instead:
// 2^y = 2^n 2^f, n = round(y), 2^f on [-1/2, 1/2] a polynomial of degree 5: the
// one of constant term 1 whose largest relative error is least (a linear
// program over the interval: 9.2e-8), its coefficients rounded to float32
// (1.1e-7; 1.7e-7 with float32 steps, below the unit's 2^-22). It costs 12 issue
// slots a value against 3, so a few pairs are all that helps: 4 x 4096 tokens of 32
// heads, d 128, took 582 + 644 thousand clocks (kRows + kKeys) at 0 of 16,
// 552 + 624 at 2, 553 + 645 at 3, 573 + 678 at 4.
#pragma once

#include "decode.cuh"
#include "prefill.cuh"

namespace gqa {

constexpr int kPsRows = 128;  // rows of a stationary and of a streamed tile
constexpr int kPsCompute = 16;
constexpr int kPsThreads = (kPsCompute + 2) * 32;
constexpr int kPsLse = 8;  // slots of the lse ring: see the producer
constexpr int kPsTmemCols = 512;
constexpr int kPsPoly = 2;  // of 16 column pairs

enum PsKind { kPsKindRows = 0, kPsKindKeys = 1 };

struct PsItem {
  int unit, pair, split, begin, n, subs, len;  // streamed tiles begin .. begin + n - 1; subs: stationary tiles with
                                               // work (the second one's S is computed in any case, and not used)
};

template <int D>
struct PsCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kPsRows * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kStreamOff = 4 * kTileBytes;  // after two slots of two stationary tiles
  static constexpr int kLseOff = kStreamOff + kStages * kTileBytes;
  static constexpr int kJoinOff = kLseOff + kPsLse * kPsRows * 4;  // float2 [item parity][t][row]
  static constexpr int kItemOff = kJoinOff + 4 * kPsRows * 8;
  static constexpr int kBarOff = kItemOff + 2 * 32;
  // st_full 2, item_full 2, item_empty 2, full, empty, s_full 4, s_free 4, lse_full, join 16, mma_done
  static constexpr int kNumBars = 6 + 2 * kStages + 8 + kPsLse + 16 + 1;
  static constexpr int kSmemBytes = kBarOff + kNumBars * 8 + 16;
};

struct PromptParams {
  float* scores;   // [B, K, S_max]
  float* nlse;     // [B * K, n_rt, 128]: -lse; -inf for a row that does not count, or sees keys at -inf alone
  float2* ml;      // key splits > 1: (m, l) [splits, B * K, n_rt, 128]
  float* part;     // row splits > 1: [splits, B * K, S_max]
  unsigned long long* queue;  // [2] this kernel's tagged work counter
  unsigned long long tag;
  const int32_t* seqlens;
  int B, T, H, K, G, S_max;
  int tile_tokens;  // tokens of a row tile, 128 / G
  int n_rt, n_kt;   // row tiles of a unit, key tiles of S_max
  int splits, items;  // of this kernel
  float scale_log2;
};

// The streamed tiles of an item. kRows: key tiles up to the pair's last row;
// kKeys: row tiles from the first query that sees the pair's first key on.
template <int kKind>
__device__ __forceinline__ PsItem ps_item(const PromptParams& p, int i) {
  PsItem it;
  const int units = p.B * p.K;
  const int tiles = kKind == kPsKindRows ? p.n_rt : p.n_kt, pairs = (tiles + 1) / 2;
  it.split = i % p.splits;
  it.unit = (i / p.splits) % units;
  const int k = i / p.splits / units;
  it.pair = kKind == kPsKindRows ? pairs - 1 - k : k;  // the longest items first
  it.subs = min(2, tiles - 2 * it.pair);
  const int len = __ldcg(p.seqlens + it.unit / p.K);
  it.len = (len < 0 || len > p.S_max) ? 0 : len;
  int first, last;
  if (kKind == kPsKindRows) {
    const int i1 = min(p.T, (2 * it.pair + 2) * p.tile_tokens) - 1;  // the pair's last token
    const int pos = it.len - p.T + i1;
    first = 0;
    last = pos < 0 ? 0 : pos / kPsRows + 1;
  } else {
    const int t0 = 2 * it.pair * kPsRows;
    const int i0 = max(0, t0 - (it.len - p.T));  // the first query that sees key t0 (and has a position >= 0)
    const bool any = t0 < it.len && i0 < p.T;
    first = any ? i0 / p.tile_tokens : 0;
    last = any ? p.n_rt : 0;
    if (t0 + kPsRows >= it.len) it.subs = 1;
  }
  const int n = last - first, per = (n + p.splits - 1) / p.splits;
  it.begin = min(last, first + it.split * per);
  it.n = min(last, it.begin + per) - it.begin;
  return it;
}

// ---- pairs of floats, one instruction for both
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(F2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// -127 .. 127 (kUpper false: up to the y given); a NaN stays one
template <bool kUpper>
__device__ __forceinline__ float clamp_exp2(float y) {
  float r;
  if (kUpper)
    asm("{\n .reg .f32 t;\n max.NaN.f32 t, %1, 0fC2FE0000;\n min.NaN.f32 %0, t, 0f42FE0000;\n}" : "=f"(r) : "f"(y));
  else
    asm("max.NaN.f32 %0, %1, 0fC2FE0000;" : "=f"(r) : "f"(y));
  return r;
}

// Operands of exp2_poly_add in constant memory, where an instruction takes them as they are: 1.5 2^23 and its
// negative, -1, then the coefficients from the highest.
__constant__ float2 kPsConst[9] = {
    {12582912.f, 12582912.f}, {-12582912.f, -12582912.f}, {-1.f, -1.f},
    {0.0013264728477224708f, 0.0013264728477224708f}, {0.009671512991189957f, 0.009671512991189957f},
    {0.05550733581185341f, 0.05550733581185341f}, {0.24022242426872253f, 0.24022242426872253f},
    {0.6931470036506653f, 0.6931470036506653f}, {1.f, 1.f}};

__device__ __forceinline__ F2 ps_const(int i) { return reinterpret_cast<const F2*>(kPsConst)[i]; }

// acc += (2^y0, 2^y1) on the FMA pipe. 2^-127 and below: 0, exactly.
template <bool kUpper>
__device__ __forceinline__ F2 exp2_poly_add(float y0, float y1, F2 acc) {
  const F2 y = f2(clamp_exp2<kUpper>(y0), clamp_exp2<kUpper>(y1));
  const F2 t = f2_add(y, ps_const(0));  // the integer nearest to y in the low bits
  const F2 f = f2_fma(f2_add(t, ps_const(1)), ps_const(2), y);
  F2 e = f2_fma(f, ps_const(3), ps_const(4));
  e = f2_fma(e, f, ps_const(5));
  e = f2_fma(e, f, ps_const(6));
  e = f2_fma(e, f, ps_const(7));
  e = f2_fma(e, f, ps_const(8));
  float t0, t1;
  f2_get(t, t0, t1);
  const float s0 = __uint_as_float((__float_as_uint(t0) << 23) + 0x3f800000u);  // 2^n
  const float s1 = __uint_as_float((__float_as_uint(t1) << 23) + 0x3f800000u);
  return f2_fma(e, f2(s0, s1), acc);
}

// Sum of 2^y over 32 columns
template <bool kUpper>
__device__ __forceinline__ float exp2_sum32(const float (&y)[32]) {
  F2 a = f2(0.f, 0.f), b = f2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    // polynomial pairs spread among the others
    if ((i * kPsPoly) % 16 < kPsPoly)
      a = exp2_poly_add<kUpper>(y[2 * i], y[2 * i + 1], a);
    else
      b = f2_add(b, f2(fast_exp2(y[2 * i]), fast_exp2(y[2 * i + 1])));
  }
  float s0, s1;
  f2_get(f2_add(a, b), s0, s1);
  return s0 + s1;
}

// kZeroRows: G does not divide 128 (a look at every tile's sums: 4 % at 7 heads a group, 4 to 8 % at 3)
template <int D, int kKind, bool kZeroRows>
__global__ void __launch_bounds__(kPsThreads, 1)
    prompt_scores_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const PromptParams p) {
  using C = PsCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* st_full = bars;                      // [2] a slot's stationary tiles landed
  uint64_t* item_full = st_full + 2;             // [2] the slot's item is written
  uint64_t* item_empty = item_full + 2;          // [2] every compute warp and the MMA warp are done with it
  uint64_t* full = item_empty + 2;               // [stages] a streamed tile landed
  uint64_t* empty = full + C::kStages;           // [stages] its MMAs finished
  uint64_t* s_full = empty + C::kStages;         // [t][2] S written
  uint64_t* s_free = s_full + 4;                 // [t][2] S read by the tile's 8 warps
  uint64_t* lse_full = s_free + 4;               // [8] kKeys: lse of a streamed tile landed
  uint64_t* join = lse_full + kPsLse;            // [slot][t][q] the upper half's sums are written
  uint64_t* mma_done = join + 16;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  PsItem* items = reinterpret_cast<PsItem*>(smem + C::kItemOff);
  static_assert(sizeof(PsItem) <= 32, "an item's slot");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_dep_wait();
  grid_dep_launch();
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle pattern assumes 1024-byte aligned tiles
    if (threadIdx.x == 0) raise_error(GQA_DEVERR_TIMEOUT);
    return;
  }
  if (kKind == kPsKindRows && blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += kPsThreads) {
      const int len = p.seqlens[b];
      if (len < 0 || len > p.S_max) raise_error(GQA_DEVERR_SEQLEN);
    }
  const int tile_rows = p.tile_tokens * p.G;  // rows of a row tile that hold queries
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&st_full[s], 1);
      mbar_init(&item_full[s], 1);
      mbar_init(&item_empty[s], kPsCompute + 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 8);
    }
    for (int s = 0; s < kPsLse; ++s) mbar_init(&lse_full[s], 1);
    for (int s = 0; s < 16; ++s) mbar_init(&join[s], 1);
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (tile_rows < kPsRows) {
    // the rows of a query tile that TMA does not write: zero, once
    const int bufs = kKind == kPsKindRows ? 4 : C::kStages;
    const int per_half = (kPsRows - tile_rows) * 8;  // 16-byte chunks
    for (int i = threadIdx.x; i < bufs * C::kHalves * per_half; i += kPsThreads) {
      const int c = i % per_half, hf = (i / per_half) % C::kHalves, s = i / per_half / C::kHalves;
      uint8_t* tile = smem + (kKind == kPsKindRows ? 0 : C::kStreamOff) + s * C::kTileBytes + hf * C::kHalfBytes;
      reinterpret_cast<uint4*>(tile + tile_rows * 128)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_shared();
  }
  if (warp == kPsCompute) {
    tmem_alloc(tmem_holder, kPsTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == kPsCompute + 1) {
    // ------------------------------------------------------- items and TMA
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      const uint64_t pol = l2_policy_evict_last();
      const uint32_t q_bytes = (uint32_t)(tile_rows * 128 * C::kHalves);
      auto load_q = [&](uint8_t* dst, const PsItem& it, int rt, uint64_t* bar) {
        const int b = it.unit / p.K, g = it.unit % p.K;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(dst + hf * C::kHalfBytes, &tm_q, hf * 64, g * p.G, b * p.T + rt * p.tile_tokens, bar, pol);
      };
      auto load_k = [&](uint8_t* dst, const PsItem& it, int kt, uint64_t* bar) {
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_2d(dst + hf * C::kHalfBytes, &tm_k, hf * 64, it.unit * p.S_max + kt * kPsRows, bar, pol);
      };
      int jt = 0;  // streamed tiles issued
      int k = 0;   // items issued
      bool ok = true;
      int item = blockIdx.x;
      while (item < p.items) {
        const int ticket = take_ticket(p.queue, p.tag);  // the next item's: its latency runs along with this one
        const PsItem it = ps_item<kKind>(p, item);
        item = ticket <= 0 ? p.items : (int)gridDim.x + ticket - 1;
        if (it.n <= 0 && (p.splits == 1 || it.len == 0)) continue;  // nothing reads what it would write
        const int slot = k & 1;
        if (k >= 2) ok = mbar_wait_bounded(&item_empty[slot], ((k >> 1) - 1) & 1);
        if (!ok) break;
        items[slot] = it;
        mbar_arrive(&item_full[slot]);
        ++k;
        if (it.n > 0) {
          uint8_t* st = smem + slot * 2 * C::kTileBytes;
          mbar_arrive_expect_tx(&st_full[slot],
                                (kKind == kPsKindRows ? q_bytes : (uint32_t)C::kTileBytes) * (uint32_t)it.subs);
          for (int t = 0; t < it.subs; ++t) {
            if (kKind == kPsKindRows)
              load_q(st + t * C::kTileBytes, it, 2 * it.pair + t, &st_full[slot]);
            else
              load_k(st + t * C::kTileBytes, it, 2 * it.pair + t, &st_full[slot]);
          }
        } else {
          mbar_arrive(&st_full[slot]);
        }
        for (int j = 0; j < it.n; ++j, ++jt) {
          const int s = jt % C::kStages;
          // kKeys: this wait is for the MMAs of tile jt - stages, which waited until every thread had given back
          // the S buffer of tile jt - stages - 2, after its last read of that tile's lse; this slot of the lse ring
          // held tile jt - 8's
          if (jt >= C::kStages) ok = mbar_wait_bounded(&empty[s], ((jt / C::kStages) - 1) & 1);
          if (!ok) break;
          uint8_t* dst = smem + C::kStreamOff + s * C::kTileBytes;
          if (kKind == kPsKindRows) {
            mbar_arrive_expect_tx(&full[s], C::kTileBytes);
            load_k(dst, it, it.begin + j, &full[s]);
          } else {
            mbar_arrive_expect_tx(&full[s], q_bytes);
            load_q(dst, it, it.begin + j, &full[s]);
            uint64_t* bar = &lse_full[jt % kPsLse];
            mbar_arrive_expect_tx(bar, kPsRows * 4);
            bulk_load(smem + C::kLseOff + (jt % kPsLse) * kPsRows * 4,
                      p.nlse + ((size_t)it.unit * p.n_rt + it.begin + j) * kPsRows, kPsRows * 4, bar);
          }
        }
        if (!ok) break;
      }
      leave_queue(p.queue, p.tag);
      if (ok) {  // no more items
        const int slot = k & 1;
        if (k >= 2) ok = mbar_wait_bounded(&item_empty[slot], ((k >> 1) - 1) & 1);
        if (ok) {
          items[slot].unit = -1;
          mbar_arrive(&item_full[slot]);
        }
      }
      // this CTA's own loads must land before the block may exit
      for (int i = max(0, k - 2); i < k; ++i) mbar_wait_bounded(&st_full[i & 1], (i >> 1) & 1);
      for (int j = max(0, jt - C::kStages); j < jt; ++j) mbar_wait_bounded(&full[j % C::kStages], (j / C::kStages) & 1);
      if (kKind == kPsKindKeys)
        for (int j = max(0, jt - kPsLse); j < jt; ++j) mbar_wait_bounded(&lse_full[j % kPsLse], (j / kPsLse) & 1);
    }
  } else if (warp == kPsCompute) {
    // -------------------------------------------------------------- MMA
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(kPsRows, kPsRows, false, false);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
    };
    auto commit = [&](uint64_t* bar) {
      if (leader) tc_commit(bar);
      __syncwarp();
    };
    int jt = 0;
    for (int k = 0;; ++k) {
      const int slot = k & 1;
      bool ok = wait_all(&item_full[slot], (k >> 1) & 1);
      if (!ok) break;
      const int unit = items[slot].unit, n = items[slot].n;
      if (unit < 0) break;
      ok = wait_all(&st_full[slot], (k >> 1) & 1);
      const uint32_t a_base = smem_u32(smem + slot * 2 * C::kTileBytes);
      for (int j = 0; ok && j < n; ++j, ++jt) {
        const int s = jt % C::kStages;
        ok = wait_all(&full[s], (jt / C::kStages) & 1);
        if (!ok) break;
        const uint32_t b_addr = smem_u32(smem + C::kStreamOff + s * C::kTileBytes);
        const int buf = jt & 1;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (jt >= 2) ok = wait_all(&s_free[2 * t + buf], ((jt >> 1) - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::kHalfBytes + (kk & 3) * 32;
              tc_mma(tmem + (uint32_t)((2 * t + buf) * kPsRows),
                     smem_desc_sw128(a_base + t * C::kTileBytes + off, 16, 1024),
                     smem_desc_sw128(b_addr + off, 16, 1024), idesc, kk > 0 ? 1u : 0u);
            }
          }
          __syncwarp();
          commit(&s_full[2 * t + buf]);
        }
        if (!ok) break;
        commit(&empty[s]);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&item_empty[slot]);
    }
    commit(mma_done);
    wait_all(mma_done, 0);
  } else {
    // ------------------------------------------------- half a row per thread
    const int t = warp >> 3, h = (warp >> 2) & 1, q = warp & 3;
    const int r = q * 32 + lane;  // row of the stationary tile
    const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(2 * t * kPsRows + h * 64);
    float2* joined = reinterpret_cast<float2*>(smem + C::kJoinOff);
    const F2 scale2 = f2(p.scale_log2, p.scale_log2);
    int jt = 0;
    for (int k = 0;; ++k) {
      const int slot = k & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&item_full[slot], (k >> 1) & 1))) break;
      const PsItem it = items[slot];
      if (it.unit < 0) break;
      bool ok = true;
      // kRows: the row's position (-1: it does not count), the warp's lowest and highest; kKeys: its key, and the
      // warp's first key's distance from the sequence's first query
      const int tok = (2 * it.pair + t) * p.tile_tokens + r / p.G;
      const int pos = (r < tile_rows && tok < p.T) ? it.len - p.T + tok : -1;
      const int pos_lo = kKind == kPsKindRows ? __reduce_min_sync(0xffffffffu, pos) : 0;
      const int pos_hi = kKind == kPsKindRows ? __reduce_max_sync(0xffffffffu, pos) : 0;
      const int key = (2 * it.pair + t) * kPsRows + r;
      const int key_off = key - lane - (it.len - p.T);
      float m = -INFINITY, l = 0.f;  // kKeys: l is the sum
      bool first = true;
      float* const score = p.scores + (size_t)it.unit * p.S_max + key;
      float before = 0.f;
      if (kKind == kPsKindKeys && h == 0 && p.splits == 1 && key < it.len) before = *score;
      for (int j = 0; j < it.n; ++j, ++jt) {
        const int buf = jt & 1;
        const uint32_t col = lane_addr + (uint32_t)(buf * kPsRows);
        // tcgen05.ld is warp-collective: every decision that guards it is warp-uniform
        bool landed = mbar_wait_bounded(&s_full[2 * t + buf], (jt >> 1) & 1);
        if (kKind == kPsKindKeys) landed = landed && mbar_wait_bounded(&lse_full[jt % kPsLse], (jt / kPsLse) & 1);
        if (!__all_sync(0xffffffffu, landed)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (kKind == kPsKindRows) {
          const int key0 = (it.begin + j) * kPsRows + h * 64;
          const int lim = pos - key0;  // columns 0 .. lim of the half are seen
          const bool masked = pos_lo - key0 < 63;
          const int chunks = min(2, (pos_hi - key0 + 32) >> 5);  // 32-column chunks that any row of the warp sees
          // sum of 2^(x - ref)
          auto pass = [&](float ref) {
            const F2 neg = f2(-ref, -ref);
            float s = 0.f;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              float x[32];
              tmem_ld32(col + c * 32, x);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 2) f2_get(f2_fma(f2(x[i], x[i + 1]), scale2, neg), x[i], x[i + 1]);
              if (masked) {
                const int last = lim - c * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i > last) x[i] = -INFINITY;
              }
              s += exp2_sum32<true>(x);
            }
            return s;
          };
          float s = 0.f;
          bool again = true;
          if (!first) {
            s = pass(m == -INFINITY ? 0.f : m);
            // the reference lies far below, or there is none (keys at -inf alone so far) and the row sees some of these
            // keys: whatever their sum against 0 is, all of them may lie below 2^-126
            again = __any_sync(0xffffffffu, !(s < 1e30f) || (m == -INFINITY && lim >= 0));
          }
          if (again) {
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              float x[32];
              tmem_ld32(col + c * 32, x);
              tc_wait_ld();
              const int last = lim - c * 32;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i <= last) top = fmaxf(top, x[i] * p.scale_log2);
            }
            const float mn = fmaxf(m, top);
            if (mn != -INFINITY) l *= fast_exp2(m - mn);  // nothing seen yet: 0
            m = mn;
            s = pass(m == -INFINITY ? 0.f : m);
          }
          first = false;
          l += s;
        } else {
          const float* ls = reinterpret_cast<const float*>(smem + C::kLseOff) + (jt % kPsLse) * kPsRows + h * 64;
          // columns from cmin on see this key: row c is token (tile's first) + c / G at position len - T + token;
          // tiles that hold tokens outside the sequence, or past its T, look at every row's lse
          const int tok0 = (it.begin + j) * p.tile_tokens;
          auto cmin_of = [&](int off) { return min(max(off - tok0, -1), kPsRows) * p.G - h * 64; };
          const int cmin = cmin_of(key_off + lane);
          bool odd = tok0 < p.T - it.len || tok0 + p.tile_tokens > p.T;
          float s;
          for (;;) {
            s = 0.f;
            const bool all = !odd && cmin_of(key_off + 31) <= 0;
#pragma unroll 1
            for (int c = max(cmin_of(key_off), 0) >> 5; c < 2; ++c) {  // from the first column that any key sees
              float x[32];
              tmem_ld32(col + c * 32, x);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const ulonglong2 zz = *reinterpret_cast<const ulonglong2*>(ls + c * 32 + i);
                f2_get(f2_fma(f2(x[i], x[i + 1]), scale2, zz.x), x[i], x[i + 1]);
                f2_get(f2_fma(f2(x[i + 2], x[i + 3]), scale2, zz.y), x[i + 2], x[i + 3]);
              }
              if (!all) {
                const int from = cmin - c * 32;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i < from) x[i] = -INFINITY;
                if (odd) {  // rows that do not count hold anything, NaN included
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (ls[c * 32 + i] == -INFINITY) x[i] = -INFINITY;
                }
              }
              s += exp2_sum32<false>(x);
            }
            // a tile's zero rows are NaN with an infinite key: the tile once more, without them
            if (!kZeroRows || odd || !__any_sync(0xffffffffu, s != s && key < it.len)) break;
            odd = true;
          }
          l += s;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[2 * t + buf]);
      }
      if (!ok) break;
      // the upper half's (m, l) to the lower half's thread of the row; the slot of this item's parity is free again
      // once both are done with the item (item_empty)
      float2* mine = joined + (slot * 2 + t) * kPsRows + r;
      uint64_t* bar = &join[8 * slot + 4 * t + q];
      if (h == 1) {
        *mine = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar, (k >> 1) & 1))) break;
        const float2 o = *mine;
        if (kKind == kPsKindRows) {
          const float M = fmaxf(m, o.x);
          // M = -inf: nothing seen, or keys at -inf (0), or NaN. A query without a weight adds nothing: L = 0 is not
          // divided by, here and in prompt_lse_kernel
          const float L = M == -INFINITY ? l + o.y : l * fast_exp2(m - M) + o.y * fast_exp2(o.x - M);
          const size_t row = ((size_t)it.unit * p.n_rt + 2 * it.pair + t) * kPsRows + r;
          if (t >= it.subs) {
            // no such tile
          } else if (p.splits == 1)
            p.nlse[row] = pos < 0 || L == 0.f ? -INFINITY : -(M + log2f(L));
          else
            p.ml[(size_t)it.split * p.B * p.K * p.n_rt * kPsRows + row] =
                pos < 0 ? make_float2(-INFINITY, 0.f) : make_float2(M, L);
        } else if (key < it.len) {
          if (p.splits == 1)
            *score = before + (l + o.y);
          else
            p.part[((size_t)it.split * p.B * p.K + it.unit) * p.S_max + key] = l + o.y;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[slot]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPsCompute) tmem_dealloc(tmem, kPsTmemCols);
}

// (m, l) of the key splits -> -lse, in order of the splits.
__global__ void prompt_lse_kernel(float* __restrict__ nlse, const float2* __restrict__ ml, long long rows, int splits) {
  grid_dep_wait();
  grid_dep_launch();
  for (long long r = blockIdx.x * (long long)blockDim.x + threadIdx.x; r < rows;
       r += (long long)gridDim.x * blockDim.x) {
    float M = -INFINITY, L = 0.f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
      const float2 v = __ldcg(&ml[s * rows + r]);
      const float mn = fmaxf(M, v.x);
      L = mn == -INFINITY ? L + v.y : L * fast_exp2(M - mn) + v.y * fast_exp2(v.x - mn);  // (-inf, 0 or NaN)
      M = mn;
    }
    nlse[r] = L == 0.f ? -INFINITY : -(M + log2f(L));
  }
}

// scores += the row splits' parts, in order.
__global__ void prompt_add_kernel(float* __restrict__ scores, const float* __restrict__ part,
                                  const int32_t* __restrict__ seqlens, int units, int K, int S_max, int splits) {
  grid_dep_wait();
  grid_dep_launch();
  const long long total = (long long)units * S_max;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int len = __ldcg(seqlens + i / S_max / K);
    if (len > S_max || i % S_max >= len) continue;
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += __ldcg(part + k * total + i);
    scores[i] += s;
  }
}

}  // namespace gqa
