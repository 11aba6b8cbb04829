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
//   kRows  x   = Q K^T: a thread owns a query row: running maximum and sum
//   kKeys  x^T = K Q^T: a thread owns a key: sum of the rows' weights, each
//          row's lse read from shared memory
// The rows of a group are taken together, r = i * G + h: a 128-row tile is
// 128 / G tokens of the G heads (fewer rows when G does not divide 128; the
// rest of the tile is zero). The stationary tile (Q or K) is loaded once per
// CTA, the other operand streams through a 2-stage ring, causal bounds drop
// tiles without work. Work items are split over keys (kRows) or rows (kKeys)
// while there are too few for the GPU; the parts are joined in a fixed order.
//
// Bound: one exponential per pair and kernel (16 per clock and SM): 1024
// clocks for a 128 x 128 tile against 512 of the MMA at d = 128.
#pragma once

#include "prefill.cuh"

namespace gqa {

constexpr int kPsRows = 128;  // rows of the stationary and of a streamed tile
constexpr int kPsThreads = 192;
constexpr int kPsStages = 2;
constexpr int kPsLse = 8;  // slots of the lse ring: see the producer
constexpr int kPsTmemCols = 256;

enum PsKind { kPsKindRows = 0, kPsKindKeys = 1 };

template <int D>
struct PsCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kPsRows * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kStreamOff = kTileBytes;
  static constexpr int kLseOff = kStreamOff + kPsStages * kTileBytes;
  static constexpr int kBarOff = kLseOff + kPsLse * kPsRows * 4;
  static constexpr int kNumBars = 1 + 2 * kPsStages + 2 + 2 + kPsLse + 1;
  // at most two CTAs per SM (their 2 x 256 TMEM columns fill the SM's 512)
  static constexpr int kNeed = kBarOff + kNumBars * 8 + 32;
  static constexpr int kSmemBytes = kNeed > 80 * 1024 ? kNeed : 80 * 1024;
};

struct PromptParams {
  float* scores;   // [B, K, S_max]
  float* lse;      // [B * K, n_rt, 128]: +inf for a row that does not count
  float2* ml;      // key splits > 1: (m, l) [splits, B * K, n_rt, 128]
  float* part;     // row splits > 1: [splits, B * K, S_max]
  const int32_t* seqlens;
  int B, T, H, K, G, S_max;
  int tile_tokens;  // tokens of a row tile, 128 / G
  int n_rt, n_kt;   // row tiles of a unit, key tiles of S_max
  int splits;       // of the streamed operand (this kernel's)
  float scale_log2;
};

// The item's streamed tiles [begin, end) of this CTA's split. kRows: key tiles
// up to the tile's last row; kKeys: row tiles from the key tile's first row on.
struct PsItem {
  int unit, tile, split, begin, end, len;
};

template <int kKind>
__device__ __forceinline__ PsItem ps_item(const PromptParams& p) {
  PsItem it;
  const int units = p.B * p.K;
  const int i = blockIdx.x;
  it.split = i % p.splits;
  it.unit = (i / p.splits) % units;
  const int k = i / p.splits / units;
  it.tile = kKind == kPsKindRows ? p.n_rt - 1 - k : k;  // the longest items first
  const int len = p.seqlens[it.unit / p.K];
  it.len = (len < 0 || len > p.S_max) ? 0 : len;
  int first, last;  // streamed tiles with work, [first, last)
  if (kKind == kPsKindRows) {
    const int i1 = min(p.T, (it.tile + 1) * p.tile_tokens) - 1;  // the tile's last token
    const int pos = it.len - p.T + i1;
    first = 0;
    last = pos < 0 ? 0 : pos / kPsRows + 1;
  } else {
    const int t0 = it.tile * kPsRows;
    const int i0 = max(0, t0 - (it.len - p.T));  // the first query that sees key t0 (and has a position >= 0)
    const bool any = t0 < it.len && i0 < p.T;
    first = any ? i0 / p.tile_tokens : 0;
    last = any ? p.n_rt : 0;
  }
  const int n = last - first, per = (n + p.splits - 1) / p.splits;
  it.begin = min(last, first + it.split * per);
  it.end = min(last, it.begin + per);
  return it;
}

template <int D, int kKind>
__global__ void __launch_bounds__(kPsThreads, 2)
    prompt_scores_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const PromptParams p) {
  using C = PsCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* st_full = bars;               // the stationary tile landed
  uint64_t* full = bars + 1;              // [2] a streamed tile landed
  uint64_t* empty = full + kPsStages;     // [2] its MMA finished
  uint64_t* s_full = empty + kPsStages;   // [2] x written to TMEM
  uint64_t* s_free = s_full + 2;          // [2] x read by all threads
  uint64_t* lse_full = s_free + 2;        // [8] kKeys: lse of a streamed tile landed
  uint64_t* mma_done = lse_full + kPsLse;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  grid_dep_wait();
  grid_dep_launch();
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle pattern assumes 1024-byte aligned tiles
    if (threadIdx.x == 0) raise_error(GQA_DEVERR_TIMEOUT);
    return;
  }
  const PsItem it = ps_item<kKind>(p);
  const int b = it.unit / p.K, g = it.unit % p.K;
  if (kKind == kPsKindRows && blockIdx.x < (unsigned)(p.B * p.K * p.splits) && it.split == 0 && g == 0 &&
      threadIdx.x == 0) {
    const int len = p.seqlens[b];
    if (len < 0 || len > p.S_max) raise_error(GQA_DEVERR_SEQLEN);
  }
  const int n_tiles = it.end - it.begin;
  const int tile_rows = p.tile_tokens * p.G;  // rows of a row tile that hold queries
  if (n_tiles <= 0) {  // the same for every thread
    if (threadIdx.x < kPsRows) {
      if (kKind == kPsKindRows) {
        const size_t r = ((size_t)it.unit * p.n_rt + it.tile) * kPsRows + threadIdx.x;
        if (p.splits == 1)
          p.lse[r] = INFINITY;
        else
          p.ml[(size_t)it.split * p.B * p.K * p.n_rt * kPsRows + r] = make_float2(-INFINITY, 0.f);
      } else if (p.splits > 1) {
        const int t = it.tile * kPsRows + threadIdx.x;
        if (t < it.len) p.part[((size_t)it.split * p.B * p.K + it.unit) * p.S_max + t] = 0.f;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(st_full, 1);
    for (int s = 0; s < kPsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 128);
    }
    for (int s = 0; s < kPsLse; ++s) mbar_init(&lse_full[s], 1);
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (tile_rows < kPsRows) {
    // the rows of a query tile that TMA does not write: zero, once
    const int bufs = kKind == kPsKindRows ? 1 : kPsStages;
    const int per_half = (kPsRows - tile_rows) * 8;  // 16-byte chunks
    for (int i = threadIdx.x; i < bufs * C::kHalves * per_half; i += kPsThreads) {
      const int c = i % per_half, hf = (i / per_half) % C::kHalves, s = i / per_half / C::kHalves;
      uint8_t* tile = smem + (kKind == kPsKindRows ? 0 : C::kStreamOff + s * C::kTileBytes) + hf * C::kHalfBytes;
      reinterpret_cast<uint4*>(tile + tile_rows * 128)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_async_shared();
  }
  if (warp == 5) {
    tmem_alloc(tmem_holder, kPsTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 4) {
    // -------------------------------------------------------------- TMA
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      const uint64_t pol = l2_policy_evict_last();
      const uint32_t q_bytes = (uint32_t)(tile_rows * 128 * C::kHalves);
      auto load_q = [&](uint8_t* dst, int rt, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, q_bytes);
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_3d(dst + hf * C::kHalfBytes, &tm_q, hf * 64, g * p.G, b * p.T + rt * p.tile_tokens, bar, pol);
      };
      auto load_k = [&](uint8_t* dst, int kt, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf)
          tma_load_2d(dst + hf * C::kHalfBytes, &tm_k, hf * 64, it.unit * p.S_max + kt * kPsRows, bar, pol);
      };
      if (kKind == kPsKindRows)
        load_q(smem, it.tile, st_full);
      else
        load_k(smem, it.tile, st_full);
      int issued = 0;
      for (int j = 0; j < n_tiles; ++j) {
        const int s = j % kPsStages;
        // kKeys: this wait is for the MMA of tile j - 2, which waited until every thread had given tile j - 4's
        // TMEM columns back; a thread does that after its last read of tile j - 5's lse, and this slot held j - 8's
        if (j >= kPsStages && !mbar_wait_bounded(&empty[s], ((j / kPsStages) - 1) & 1)) break;
        uint8_t* dst = smem + C::kStreamOff + s * C::kTileBytes;
        if (kKind == kPsKindRows) {
          load_k(dst, it.begin + j, &full[s]);
        } else {
          load_q(dst, it.begin + j, &full[s]);
          uint64_t* bar = &lse_full[j % kPsLse];
          mbar_arrive_expect_tx(bar, kPsRows * 4);
          bulk_load(smem + C::kLseOff + (j % kPsLse) * kPsRows * 4,
                    p.lse + ((size_t)it.unit * p.n_rt + it.begin + j) * kPsRows, kPsRows * 4, bar);
        }
        ++issued;
      }
      // this CTA's own loads must land before the block may exit
      mbar_wait_bounded(st_full, 0);
      for (int j = max(0, issued - kPsStages); j < issued; ++j)
        mbar_wait_bounded(&full[j % kPsStages], (j / kPsStages) & 1);
      if (kKind == kPsKindKeys)
        for (int j = max(0, issued - kPsLse); j < issued; ++j)
          mbar_wait_bounded(&lse_full[j % kPsLse], (j / kPsLse) & 1);
    }
  } else if (warp == 5) {
    // -------------------------------------------------------------- MMA
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(kPsRows, kPsRows, false, false);
    const uint32_t a_addr = smem_u32(smem);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
    };
    auto commit = [&](uint64_t* bar) {
      if (leader) tc_commit(bar);
      __syncwarp();
    };
    bool ok = wait_all(st_full, 0);
    for (int j = 0; ok && j < n_tiles; ++j) {
      const int s = j % kPsStages;
      ok = wait_all(&full[s], (j / kPsStages) & 1);
      if (ok && j >= 2) ok = wait_all(&s_free[j & 1], ((j >> 1) - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t b_addr = smem_u32(smem + C::kStreamOff + s * C::kTileBytes);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kHalfBytes + (kk & 3) * 32;
          tc_mma(tmem + (uint32_t)((j & 1) * kPsRows), smem_desc_sw128(a_addr + off, 16, 1024),
                 smem_desc_sw128(b_addr + off, 16, 1024), idesc, kk > 0 ? 1u : 0u);
        }
      }
      __syncwarp();
      commit(&s_full[j & 1]);
      commit(&empty[s]);
    }
    commit(mma_done);
    wait_all(mma_done, 0);
  } else {
    // -------------------------------------------------- one thread per row
    const int r = threadIdx.x;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    bool ok = true;
    float m = -INFINITY, l = 0.f;  // kRows
    float acc = 0.f;               // kKeys
    const int tok = it.tile * p.tile_tokens + r / p.G;  // kRows: the row's query
    const int pos = (r < tile_rows && tok < p.T) ? it.len - p.T + tok : -1;
    const int key = it.tile * kPsRows + r;  // kKeys
    for (int j = 0; j < n_tiles; ++j) {
      // tcgen05.ld is warp-collective: every decision that guards it is warp-uniform
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&s_full[j & 1], (j >> 1) & 1)) ||
          (kKind == kPsKindKeys &&
           !__all_sync(0xffffffffu, mbar_wait_bounded(&lse_full[j % kPsLse], (j / kPsLse) & 1)))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t col = lane_addr + (uint32_t)((j & 1) * kPsRows);
      if (kKind == kPsKindRows) {
        const int lim = pos - (it.begin + j) * kPsRows;  // columns 0 .. lim are seen
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float x[64];
          {
            float a[32], c[32];
            tmem_ld32(col + hf * 64, a);
            tmem_ld32(col + hf * 64 + 32, c);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = a[i] * p.scale_log2;
              x[32 + i] = c[i] * p.scale_log2;
            }
          }
          if (hf == 1) {
            tc_fence_before();
            mbar_arrive(&s_free[j & 1]);
          }
          if (lim < hf * 64 + 63) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (hf * 64 + i > lim) x[i] = -INFINITY;
          }
          const float mn = fmaxf(m, max64(x));
          const float ref = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every term is 2^-inf
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            s0 += fast_exp2(x[i] - ref);
            s1 += fast_exp2(x[i + 1] - ref);
          }
          l = l * fast_exp2(m - ref) + (s0 + s1);
          m = mn;
        }
      } else {
        const float* ls = reinterpret_cast<const float*>(smem + C::kLseOff) + (j % kPsLse) * kPsRows;
        // columns from cmin on see this key: row c is token (tile's first) + c / G at position len - T + token
        const int cmin = (key - (it.len - p.T) - (it.begin + j) * p.tile_tokens) * p.G;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int hf = 0; hf < 4; ++hf) {
          float x[32];
          tmem_ld32(col + hf * 32, x);
          tc_wait_ld();
          if (hf == 3) {
            tc_fence_before();
            mbar_arrive(&s_free[j & 1]);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 z = *reinterpret_cast<const float4*>(ls + hf * 32 + i);
            const float e0 = fast_exp2(x[i] * p.scale_log2 - z.x), e1 = fast_exp2(x[i + 1] * p.scale_log2 - z.y);
            const float e2 = fast_exp2(x[i + 2] * p.scale_log2 - z.z), e3 = fast_exp2(x[i + 3] * p.scale_log2 - z.w);
            const int c = hf * 32 + i;
            s0 += (c >= cmin && z.x != INFINITY) ? e0 : 0.f;
            s1 += (c + 1 >= cmin && z.y != INFINITY) ? e1 : 0.f;
            s0 += (c + 2 >= cmin && z.z != INFINITY) ? e2 : 0.f;
            s1 += (c + 3 >= cmin && z.w != INFINITY) ? e3 : 0.f;
          }
        }
        acc += s0 + s1;
      }
    }
    if (ok) {
      if (kKind == kPsKindRows) {
        const size_t row = ((size_t)it.unit * p.n_rt + it.tile) * kPsRows + r;
        if (p.splits == 1)
          p.lse[row] = pos < 0 ? INFINITY : m + log2f(l);
        else
          p.ml[(size_t)it.split * p.B * p.K * p.n_rt * kPsRows + row] =
              pos < 0 ? make_float2(-INFINITY, 0.f) : make_float2(m, l);
      } else if (key < it.len) {
        if (p.splits == 1)
          p.scores[(size_t)it.unit * p.S_max + key] += acc;
        else
          p.part[((size_t)it.split * p.B * p.K + it.unit) * p.S_max + key] = acc;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kPsTmemCols);
}

// (m, l) of the key splits -> lse, in order of the splits.
__global__ void prompt_lse_kernel(float* __restrict__ lse, const float2* __restrict__ ml, long long rows, int splits) {
  grid_dep_wait();
  grid_dep_launch();
  for (long long r = blockIdx.x * (long long)blockDim.x + threadIdx.x; r < rows;
       r += (long long)gridDim.x * blockDim.x) {
    float M = -INFINITY, L = 0.f;
    for (int s = 0; s < splits; ++s) M = fmaxf(M, __ldcg(&ml[s * rows + r].x));
    for (int s = 0; s < splits; ++s) {
      const float2 v = __ldcg(&ml[s * rows + r]);
      if (v.y != 0.f) L += v.y * fast_exp2(v.x - M);
    }
    lse[r] = L == 0.f ? INFINITY : M + log2f(L);
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
    const int len = __ldg(seqlens + i / S_max / K);
    if (len > S_max || i % S_max >= len) continue;
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += __ldcg(part + k * total + i);
    scores[i] += s;
  }
}

}  // namespace gqa
