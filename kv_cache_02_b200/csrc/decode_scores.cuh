// gqa_decode_scores: the decode of decode.cuh, and each cached row's share of
// the attention added to its score.
//
//   scores[b, g, t] += sum_{h in group} 2^(x[h, t] - M[h]) / L[h]
//
// with x the scaled scores in log2 units and (M, L) the softmax's maximum and
// sum over all of the sequence's keys. A row's weight is not known before the
// last split's maximum is, so the decode kernel stores its scaled scores
// (float32: a weight is as exact as its exponent), and a second kernel joins
// the splits: their outputs, and the scores as weights. Reading K again
// instead would cost 2 d bytes a key; the scores are 8 G bytes a key written
// and read back, mostly in L2.
//
// Measured, in a graph: 8 x 8192 keys of 32 and 8 heads, d 128: 52 us
// (gqa_decode: 47; the bytes at a copy's rate: 42); one sequence of 131072 keys,
// 64 and 8 heads: 102 us (86; 83), the join of 33 MB of scores included. Larger
// groups pay for their scores (8 G bytes a key) and for the tile of every head
// slice: 64 heads over 131072 keys of 4, 2 and 1 KV heads 85, 92 and 121 us
// (gqa_decode 59, 55 and 20).
#pragma once

#include "decode.cuh"

namespace gqa {

struct ScoresParams {
  float* x;       // [B * H, x_stride] scaled scores
  float* scores;  // [B, K, S_max]
  int x_stride;   // S_max rounded up to 4
};

// warp_tile of decode.cuh, storing the scaled scores of the warp's keys: xa, xb
// are the lane's two heads' scores of key kb (null: no such head).
template <int D>
__device__ __forceinline__ void warp_tile_scores(WarpState<D>& st, const uint32_t (&qf)[D / 16][2],
                                                 uint32_t stage_addr, int kb, int rows, int lane, float scale_log2,
                                                 float* xa, float* xb) {
  using C = DecCfg<D>;
  const uint32_t k_base = stage_addr;
  const uint32_t v_base = stage_addr + C::kTileBytes;
  const int k_row = kb + (lane & 7) + ((lane >> 3) & 1) * 8;
  const int k_col8 = lane >> 4;
  const int v_row = kb + (lane & 7) + (lane >> 4) * 8;
  const int v_col8 = (lane >> 3) & 1;

  float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const int chunk = ks * 2 + k_col8;
    const uint32_t addr = k_base + (chunk >> 3) * C::kHalfBytes + sw128(k_row, chunk & 7);
    uint32_t a0, a1, a2, a3;
    ldmatrix_x4(addr, a0, a1, a2, a3);
    mma_bf16_16816(c, a0, a1, a2, a3, qf[ks][0], qf[ks][1]);
  }

  const int key0 = kb + (lane >> 2);
  const bool v0 = key0 < rows, v1 = key0 + 8 < rows;
  const float x0 = v0 ? c[0] * scale_log2 : -INFINITY;
  const float x1 = v0 ? c[1] * scale_log2 : -INFINITY;
  const float x2 = v1 ? c[2] * scale_log2 : -INFINITY;
  const float x3 = v1 ? c[3] * scale_log2 : -INFINITY;
  const int at = lane >> 2;
  if (xa != nullptr) {
    if (v0) xa[at] = x0;
    if (v1) xa[at + 8] = x2;
  }
  if (xb != nullptr) {
    if (v0) xb[at] = x1;
    if (v1) xb[at + 8] = x3;
  }
  float mx_a = fmaxf(x0, x2), mx_b = fmaxf(x1, x3);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
    mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
  }
  const float mn_a = fmaxf(st.m_a, mx_a), mn_b = fmaxf(st.m_b, mx_b);
  // keys at -inf alone so far: they weigh nothing, against any finite reference
  const float r_a = mn_a == -INFINITY ? 0.f : mn_a, r_b = mn_b == -INFINITY ? 0.f : mn_b;
  const float al_a = fast_exp2(st.m_a - r_a), al_b = fast_exp2(st.m_b - r_b);
  st.m_a = mn_a;
  st.m_b = mn_b;
  const float p0 = fast_exp2(x0 - r_a), p1 = fast_exp2(x1 - r_b);
  const float p2 = fast_exp2(x2 - r_a), p3 = fast_exp2(x3 - r_b);
  st.l_a = st.l_a * al_a + p0 + p2;
  st.l_b = st.l_b * al_b + p1 + p3;
#pragma unroll
  for (int md = 0; md < D / 16; ++md) {
    st.o[md][0] *= al_a;
    st.o[md][1] *= al_b;
    st.o[md][2] *= al_a;
    st.o[md][3] *= al_b;
  }

  // P as two bfloat16 terms, off by 2^-15 of it: one would be off by 2^-9, as much as the output's own rounding, and
  // the second costs 1 % (8 x 8192 keys: 51.5 us in a graph for 50.9). The first is the value below the one that P
  // cut off gives, so that the second is above 0 too: neither makes NaN of an infinite value.
  auto below = [](float p) { return max(__float_as_uint(p), 0x10000u) - 0x10000u; };
  auto first = [&](float lo, float hi) { return __byte_perm(below(lo), below(hi), 0x7632); };
  auto rest = [](uint32_t h, float lo, float hi) {
    return pack_bf16x2(lo - __uint_as_float(h << 16), hi - __uint_as_float(h & 0xffff0000u));
  };
  const uint32_t h0 = first(p0, p1), h1 = first(p2, p3);
  const uint32_t pb0 = movmatrix_trans(h0), pb1 = movmatrix_trans(h1);
  const uint32_t pl0 = movmatrix_trans(rest(h0, p0, p1)), pl1 = movmatrix_trans(rest(h1, p2, p3));
  uint32_t mask_lo = 0xffffffffu, mask_hi = 0xffffffffu;
  if (kb + 16 > rows) {
    const int lim = rows - kb;
    const int kk = 2 * (lane & 3);
    mask_lo = (kk < lim ? 0x0000ffffu : 0u) | (kk + 1 < lim ? 0xffff0000u : 0u);
    mask_hi = (kk + 8 < lim ? 0x0000ffffu : 0u) | (kk + 9 < lim ? 0xffff0000u : 0u);
  }
#pragma unroll
  for (int md = 0; md < D / 16; ++md) {
    const int chunk = md * 2 + v_col8;
    const uint32_t addr = v_base + (chunk >> 3) * C::kHalfBytes + sw128(v_row, chunk & 7);
    uint32_t a0, a1, a2, a3;
    ldmatrix_x4_trans(addr, a0, a1, a2, a3);
    a0 &= mask_lo, a1 &= mask_lo, a2 &= mask_hi, a3 &= mask_hi;
    mma_bf16_16816(st.o[md], a0, a1, a2, a3, pb0, pb1);
    mma_bf16_16816(st.o[md], a0, a1, a2, a3, pl0, pl1);
  }
}

// End of a work item: as item_epilogue, and (m, l) of every split is kept,
// the only split's too.
template <int D>
__device__ __forceinline__ void scores_epilogue(const DecodeParams& p, const ItemCoord& c, const WarpState<D>& st,
                                                float* merge, bool single, int tid, int warp, int lane) {
  __nv_bfloat16* out_row = static_cast<__nv_bfloat16*>(p.out) + ((size_t)c.b * p.H + c.h0) * D;
  consumer_bar();
  stash_warp_state<D>(merge, st, warp, lane);
  consumer_bar();
  const size_t part = ((size_t)c.unit * p.nsplit + c.split) * p.G + (size_t)c.hsl * kDecHeadsPerCta;
  for (int i = tid; i < c.nh * D; i += kDecConsumerWarps * 32) {
    const int h = i / D, dim = i % D;
    float M, L, O;
    merged<D>(merge, h, dim, M, L, O);
    if (M == -INFINITY) {  // every key of the item is at -inf, or NaN: 0, or NaN
      L = 0.f;
      for (int w = 0; w < kDecConsumerWarps; ++w) L += merge[(kDecConsumerWarps + w) * kDecHeadsPerCta + h];
      O = L;
    }
    if (single)
      out_row[i] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);  // keys at -inf alone: zeros, as without keys
    else
      p.ws_o[(part + h) * D + dim] = O;
    if (dim == 0) p.ws_ml[part + h] = make_float2(M, L);
  }
}

// Producer of a contiguous bf16 cache (one thread): work items from the
// counter, their tiles through the ring, then a record that ends the
// consumers' loop. As in decode_bf16_kernel.
template <int D>
__device__ __forceinline__ void produce_contiguous(const DecodeParams& p, uint8_t* smem, StageInfo* info,
                                                   uint64_t* full, uint64_t* empty, const CUtensorMap* tm_k64,
                                                   const CUtensorMap* tm_v64, const CUtensorMap* tm_k16,
                                                   const CUtensorMap* tm_v16) {
  using C = DecCfg<D>;
  const uint64_t policy = l2_policy_evict_first();
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
  int it = 0;
  bool ok = true;
  for (int k = 0;; ++k) {
    const int ticket = k == 0 ? 1 : take_ticket(p.ws_queue, p.tag);
    const int item = k == 0 ? (int)blockIdx.x : (int)gridDim.x + ticket - 1;
    if (ticket <= 0 || item >= p.nitems) break;
    const ItemCoord c = item_coord(p, item);
    const int raw = __ldcg(p.seqlens + c.b);
    const int len = valid_len(raw, p.S_max);
    if (c.g == 0 && c.split == 0 && c.hsl == 0 && len != raw) raise_error(GQA_DEVERR_SEQLEN);
    const int t_begin = c.split * p.chunk;
    const int t_end = min(len, t_begin + p.chunk);
    if (t_begin >= t_end) {
      if (c.split == 0) {  // an empty sequence: zeros for this item's heads
        uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)c.b * p.H + c.h0) * D);
        for (int i = 0; i < c.nh * D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const int ntiles = (t_end - t_begin + kDecTileKeys - 1) / kDecTileKeys;
    for (int tt = 0; tt < ntiles && ok; ++tt, ++it) {
      const int s = it % C::kStages;
      const int t0 = t_begin + tt * kDecTileKeys;
      const int rows = min(kDecTileKeys, t_end - t0);
      if (it >= C::kStages) ok = mbar_wait_bounded(&empty[s], ((it / C::kStages) - 1) & 1);
      if (!ok) break;
      info[s] = StageInfo{item, rows,
                          (tt == 0 ? kTileFirst : 0) | (tt == ntiles - 1 ? kTileLast : 0) |
                              (len <= p.chunk ? kUnitSingleSplit : 0),
                          -1};
      issue_tile<D>(smem + s * C::kStageBytes, &full[s], tm_k64, tm_v64, tm_k16, tm_v16, c.unit * p.S_max + t0, rows,
                    policy);
    }
    if (!ok) break;
  }
  leave_queue(p.ws_queue, p.tag);
  if (ok) {
    const int s = it % C::kStages;
    if (it >= C::kStages) ok = mbar_wait_bounded(&empty[s], ((it / C::kStages) - 1) & 1);
    if (ok) {
      info[s] = StageInfo{-1, 0, 0, 0};
      mbar_arrive(&full[s]);
      ++it;
    }
  }
  for (int j = max(0, it - C::kStages); j < it; ++j) mbar_wait_bounded(&full[j % C::kStages], (j / C::kStages) & 1);
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kDecThreads, 2)
    decode_scores_kernel(const __grid_constant__ CUtensorMap tm_k64, const __grid_constant__ CUtensorMap tm_v64,
                         const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const DecodeParams p, const ScoresParams sp) {
  using C = DecCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + C::kMergeOff);
  StageInfo* info = reinterpret_cast<StageInfo*>(smem + C::kInfoOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzle pattern needs 1024-byte aligned stages
    grid_dep_wait();
    if (threadIdx.x == 0) raise_error(GQA_DEVERR_TIMEOUT);
    return;
  }
  // before the grid dependency: barriers, descriptors and an L2 warm-up of
  // the first work item's rows, as in decode_bf16_kernel
  int spec_first = 0;
  if (!kPaged && warp == kDecConsumerWarps && lane == 0) {
    prefetch_tensormap(&tm_k64);
    prefetch_tensormap(&tm_v64);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    if ((int)blockIdx.x < p.nitems) spec_first = __ldcg(p.seqlens + item_coord(p, blockIdx.x).b);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kDecConsumerWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (!kPaged && warp == kDecConsumerWarps && lane == 0 && (int)blockIdx.x < p.nitems)
    warm_first_item<D * C::kElt>(p, item_coord(p, blockIdx.x), spec_first, kDecWarmKeys);
  if (kPaged && warp == kDecConsumerWarps && (int)blockIdx.x < p.nitems) {
    const ItemCoord c0 = item_coord(p, blockIdx.x);
    warm_first_item_paged<D>(p, c0, __ldcg(p.seqlens + c0.b), kDecWarmKeys, lane);
  }
  grid_dep_wait();
  grid_dep_launch();

  if (warp == kDecConsumerWarps) {
    if constexpr (kPaged)
      produce_paged<D>(p, smem, info, full, empty, &tm_k64, &tm_v64, &tm_k, &tm_v, lane);
    else if (lane == 0)
      produce_contiguous<D>(p, smem, info, full, empty, &tm_k64, &tm_v64, &tm_k, &tm_v);
    return;
  }

  const int tid = threadIdx.x;
  const int kb = warp * 16;
  uint32_t qf[D / 16][2];
  int t0 = 0;  // key of the tile's first row
  WarpState<D> st;
  ItemCoord cur{};
  for (int it = 0;; ++it) {
    const int s = it % C::kStages;
    if (!mbar_wait_bounded(&full[s], (it / C::kStages) & 1)) break;
    const StageInfo si = info[s];
    if (si.item < 0) break;
    if (si.flags & kTileFirst) {
      cur = item_coord(p, si.item);
      load_q_frag<D>(qf, static_cast<const __nv_bfloat16*>(p.q) + ((size_t)cur.b * p.H + cur.h0) * D, lane, cur.nh);
      st.reset();
      t0 = cur.split * p.chunk;
    }
    if (kb < si.rows) {
      const int h = 2 * (lane & 3);
      float* x = sp.x + ((size_t)cur.b * p.H + cur.h0 + h) * sp.x_stride + t0 + kb;
      warp_tile_scores<D>(st, qf, smem_u32(smem + s * C::kStageBytes), kb, si.rows, lane, p.scale_log2,
                          h < cur.nh ? x : nullptr, h + 1 < cur.nh ? x + sp.x_stride : nullptr);
    }
    t0 += kDecTileKeys;
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (si.flags & kTileLast)
      scores_epilogue<D>(p, cur, st, merge, (si.flags & kUnitSingleSplit) != 0, tid, warp, lane);
  }
}

// The join. A CTA takes 4 Q rows a thread of one unit. Its warps first join the
// splits' (m, l) of the group's heads; then a thread adds up the heads'
// weights of its rows, in order of the heads, and the unit's output columns
// are shared out among the unit's CTAs, a CTA's threads over the splits of its
// columns (summed in a fixed order). Latency bounds it: all that does not
// depend on (m, l) is asked for first, the scores to be added to into L2 (their
// values in registers would make them spill). Q = 2 where the CTAs of Q = 1
// would not all be resident, 592 at a time: whole calls in a graph at Q = 1 and
// 2, by CTAs of Q = 1: 256 31.9 and 34.1 us, 512 50.5 and 52.4, 576 54.9 and
// 57.0, 608 68.2 and 68.4, 640 64.0 and 63.3, 1024 (131072 keys of 8 heads)
// 107.7 and 102.2, 2048 213 and 206.
constexpr int kAccThreads = 256;
constexpr int kAccHeads = 64;  // heads whose (M, 1 / L) are held at a time
// float4 of scores that a thread asks for at once (512 and 1024 CTAs: 50.5 and 102 us; two 50.8 and 100, eight, which
// spill, 54.2 and 106)
constexpr int kAccFlight = 4;

template <int D, int Q>
__global__ void __launch_bounds__(kAccThreads, 4)
    scores_finish_kernel(const DecodeParams p, const ScoresParams sp, int chunks) {
  __shared__ float2 ml[kAccHeads];
  __shared__ float4 red[kAccThreads];
  constexpr int kAccKeys = 4 * Q * kAccThreads, kAccBatch = kAccFlight / Q;
  const int unit = blockIdx.x / chunks, part = blockIdx.x % chunks;
  const int b = unit / p.K, g = unit % p.K;
  const int k0 = part * kAccKeys;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int len = valid_len(p.seqlens[b], p.S_max);
  const int n = min(kAccKeys, len - k0);
  if (n <= 0) return;
  const int ns = (len + p.chunk - 1) / p.chunk;
  const int active = (len + kAccKeys - 1) / kAccKeys;  // CTAs of the unit that have rows
  // the output columns of this CTA, four dims each
  const int cols = p.G * (D / 4), per = (cols + active - 1) / active;
  const float* x0 = sp.x + ((size_t)b * p.H + (size_t)g * p.G) * sp.x_stride + k0 + 4 * tid;
  const float2* unit_ml = p.ws_ml + (size_t)unit * p.nsplit * p.G;
  const float4* unit_o = reinterpret_cast<const float4*>(p.ws_o + (size_t)unit * p.nsplit * p.G * D);
  // this thread's rows of the scores
  float* const dst = sp.scores + (size_t)unit * p.S_max + k0 + 4 * tid;
  constexpr int kNext = 4 * kAccThreads;  // rows between a thread's quads
  bool quad[Q];
  float4 sum[Q];
#pragma unroll
  for (int u = 0; u < Q; ++u) {
    quad[u] = n - 4 * tid - u * kNext >= 4 && (p.S_max & 3) == 0;
    sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (quad[u]) asm volatile("prefetch.global.L2 [%0];" ::"l"(__cvta_generic_to_global(dst + u * kNext)));
  }
  for (int h0 = 0; h0 < p.G; h0 += kAccHeads) {
    const int nh = min(kAccHeads, p.G - h0);
    float4 x[Q][kAccBatch];
    auto ask = [&](int h) {  // rows from n on hold anything: their sums are not used
#pragma unroll
      for (int u = 0; u < Q; ++u)
#pragma unroll
        for (int i = 0; i < kAccBatch; ++i)
          if (h + i < nh && n - 4 * tid - u * kNext > 0)
            x[u][i] = __ldcg(reinterpret_cast<const float4*>(x0 + (size_t)(h0 + h + i) * sp.x_stride + u * kNext));
    };
    ask(0);
    // columns of heads h0 .. h0 + nh - 1, `width` at a time: a power of two, so that as many threads as possible
    // share the splits
    const int c0 = max(part * per, h0 * (D / 4)), c1 = min(min(part * per + per, cols), (h0 + nh) * (D / 4));
    int width = 1;
    while (width < min(c1 - c0, kAccThreads)) width *= 2;
    const int slots = kAccThreads / width;
    const int cc = tid % width, slot = tid / width;
    if (h0 > 0) __syncthreads();
    for (int h = warp; h < nh; h += kAccThreads / 32) {
      const float2* ptr = unit_ml + h0 + h;
      float M = -INFINITY, L = 0.f;
#pragma unroll 4
      for (int s = lane; s < ns; s += 32) {
        const float2 v = __ldcg(&ptr[(size_t)s * p.G]);
        const float mn = fmaxf(M, v.x);
        L = mn == -INFINITY ? L + v.y : L * fast_exp2(M - mn) + v.y * fast_exp2(v.x - mn);  // (-inf, 0 or NaN)
        M = mn;
      }
      float top = M;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      L = M == -INFINITY ? L : L * fast_exp2(M - top);  // a lane without splits holds 0
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
      // L = 0: keys at -inf alone, which weigh nothing against any finite maximum
      if (lane == 0) ml[h] = L == 0.f ? make_float2(0.f, 0.f) : make_float2(top, 1.f / L);
    }
    __syncthreads();
    for (int h = 0; h < nh; h += kAccBatch) {
      if (h > 0) ask(h);
#pragma unroll
      for (int i = 0; i < kAccBatch; ++i) {
        if (h + i < nh) {
          const float2 z = ml[h + i];
#pragma unroll
          for (int u = 0; u < Q; ++u) {
            sum[u].x = fmaf(fast_exp2(x[u][i].x - z.x), z.y, sum[u].x);
            sum[u].y = fmaf(fast_exp2(x[u][i].y - z.x), z.y, sum[u].y);
            sum[u].z = fmaf(fast_exp2(x[u][i].z - z.x), z.y, sum[u].z);
            sum[u].w = fmaf(fast_exp2(x[u][i].w - z.x), z.y, sum[u].w);
          }
        }
      }
    }
    if (ns > 1) {
      for (int c = c0; c < c1; c += width) {
        const int col = c + cc;
        const int h = col / (D / 4);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (col < c1) {
          const float top = ml[h - h0].x;
          const float4* src = unit_o + col;  // column col of split 0: head h, dims 4 (col - h D / 4)
#pragma unroll(4 / Q)
          for (int s = slot; s < ns; s += slots) {
            const float f = fast_exp2(__ldcg(&unit_ml[(size_t)s * p.G + h].x) - top);
            const float4 v = __ldcg(src + (size_t)s * cols);
            o.x = fmaf(v.x, f, o.x);
            o.y = fmaf(v.y, f, o.y);
            o.z = fmaf(v.z, f, o.z);
            o.w = fmaf(v.w, f, o.w);
          }
        }
        // the slots of a column: over the lanes of a warp, then over warps
        for (int off = 16; off >= width; off >>= 1) {
          o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
          o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
          o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
          o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
        }
        red[tid] = o;
        __syncthreads();
        if (slot == 0 && col < c1) {
          const int step = max(width, 32);
          for (int t = tid + step; t < kAccThreads; t += step) {
            const float4 v = red[t];
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
          }
          const float inv = ml[h - h0].y;
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + ((size_t)b * p.H + g * p.G) * D + col * 4) =
              make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        }
        __syncthreads();
      }
    }
  }
#pragma unroll
  for (int u = 0; u < Q; ++u) {
    if (quad[u]) {
      float4 acc = *reinterpret_cast<const float4*>(dst + u * kNext);
      acc.x += sum[u].x, acc.y += sum[u].y, acc.z += sum[u].z, acc.w += sum[u].w;
      *reinterpret_cast<float4*>(dst + u * kNext) = acc;
    } else {
      const float a[4] = {sum[u].x, sum[u].y, sum[u].z, sum[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n - 4 * tid - u * kNext) dst[u * kNext + j] += a[j];
    }
  }
}

}  // namespace gqa
