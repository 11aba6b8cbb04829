// Host side of include/gqa_cache.h: argument checks, launch plans and
// workspaces. Part of gqa_lib.cu, whose helpers it uses.
#pragma once

namespace {

PagedCache paged_cache(const int32_t* table, int num_blocks, int block_size, int max_blocks) {
  PagedCache pc;
  pc.table = table;
  pc.num_blocks = num_blocks;
  pc.block_size = block_size;
  pc.max_blocks = max_blocks;
  return pc;
}

// The workspace sizes that callers ask for: the most that any batch of up to B sequences takes (size(b, SMs), 0 where
// there is no plan), so that a buffer made for the largest batch serves every smaller one. A smaller batch may take
// more: its work is split further. From 16 sequences per SM on no plan splits anything (the most that one aims at are
// 12 work items per SM), and sizes only grow.
template <typename Size>
size_t most_over_batches(int B, Size size) {
  const int sms = sm_count(current_device());
  size_t most = size(B, sms);
  if (most == 0) return 0;
  for (int b = std::min(B, 16 * sms) - 1; b > 0; --b) most = std::max(most, size(b, sms));
  return most;
}

// ----------------------------------------------------------------------------
// gqa_qk_norm_rope

template <typename T, int D>
int launch_norm_rope(const gqa::NormRopeParams& p0, bool interleaved, int sms, cudaStream_t st) {
  constexpr int LPR = D / 8;
  gqa::NormRopeParams p = p0;
  const long long tokens = (long long)p.B * p.T;
  const int rows = p.H + p.K + (p.v_cache ? p.K : 0);
  constexpr int R = 4;
  // few tokens: one row per lane group; enough for every SM's threads four times over: R rows, so that one table
  // row, one position and one address calculation serve them
  const bool many = tokens * rows * LPR >= (long long)R * sms * 2048;
  p.chunks = many ? (rows + R - 1) / R : rows;
  const long long groups = tokens * p.chunks;
  if (groups * LPR >= (1ll << 31)) return GQA_ERR_SHAPE;
  const unsigned grid = (unsigned)((groups * LPR + gqa::kNrThreads - 1) / gqa::kNrThreads);
  auto run = [&](auto kernel) { return gqa::launch_kernel(kernel, grid, gqa::kNrThreads, 0, st, true, p); };
  if (!many)
    return interleaved ? run(gqa::qk_norm_rope_kernel<T, D, true, 1>) : run(gqa::qk_norm_rope_kernel<T, D, false, 1>);
  return interleaved ? run(gqa::qk_norm_rope_kernel<T, D, true, R>) : run(gqa::qk_norm_rope_kernel<T, D, false, R>);
}

int norm_rope_impl(void* q_out, void* k_out, void* k_cache, void* v_cache, int32_t* row_pos, const void* q,
                   const void* k, const void* v, const void* q_weight, const void* k_weight, const float* rope,
                   const int32_t* positions, const int32_t* rows, int B, int T, int H, int K, int S_max, int d,
                   int64_t q_stride, int64_t k_stride, int64_t v_stride, int rotary_dim, int max_pos, int interleaved,
                   float eps, gqa_dtype dtype, gqa_stream_t stream, const PagedCache* pc) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || H <= 0 || K <= 0 || rotary_dim < 0 || !(eps >= 0.f)) return GQA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || H % K != 0 || rotary_dim > d || rotary_dim % 16 != 0) return GQA_ERR_SHAPE;
  if ((k_cache == nullptr) != (v_cache == nullptr)) return GQA_ERR_INVALID_ARG;
  const bool cached = k_cache != nullptr || row_pos != nullptr;
  if (cached && S_max <= 0) return GQA_ERR_INVALID_ARG;
  if (cached && T > S_max) return GQA_ERR_SHAPE;
  if (rotary_dim > 0 && max_pos <= 0) return GQA_ERR_INVALID_ARG;
  const int vec = dtype == GQA_F32 ? 4 : 8;
  const int64_t qw = (int64_t)H * d, kw = (int64_t)K * d;
  if (q_stride < qw || k_stride < kw || q_stride % vec != 0 || k_stride % vec != 0) return GQA_ERR_SHAPE;
  if (k_cache && (v_stride < kw || v_stride % vec != 0)) return GQA_ERR_SHAPE;
  if (B == 0 || T == 0) return GQA_OK;
  if (!q_out || !q || !k || (k_cache && !v)) return GQA_ERR_INVALID_ARG;
  if ((rotary_dim > 0 && (!rope || !positions)) || (row_pos && !positions)) return GQA_ERR_INVALID_ARG;
  if (cached && !rows) return GQA_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(rope))
    return GQA_ERR_ALIGN;
  gqa::NormRopeParams p{};
  p.q = q;
  p.k = k;
  p.v = k_cache ? v : nullptr;
  p.q_out = q_out;
  p.k_out = k_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.row_pos = row_pos;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.rope = rope;
  p.positions = positions;
  p.rows = rows;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.B = B;
  p.T = T;
  p.H = H;
  p.K = K;
  p.S_max = S_max;
  p.rotary_dim = rotary_dim;
  p.max_pos = max_pos;
  p.eps = eps;
  if (pc) {
    p.block_table = pc->table;
    p.num_blocks = pc->num_blocks;
    p.block_size = pc->block_size;
    p.max_blocks = pc->max_blocks;
  }
  const int sms = sm_count(current_device());
  const bool il = interleaved != 0;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == GQA_BF16)
    return d == 128 ? launch_norm_rope<__nv_bfloat16, 128>(p, il, sms, st)
                    : launch_norm_rope<__nv_bfloat16, 64>(p, il, sms, st);
  return d == 128 ? launch_norm_rope<float, 128>(p, il, sms, st) : launch_norm_rope<float, 64>(p, il, sms, st);
}

// ----------------------------------------------------------------------------
// gqa_decode_scores

struct ScoresPlan {
  DecodePlan pl;
  size_t ml_off = 0, queue_off = 0, x_off = 0, bytes = 0;
};

// false: no plan (a shape that gqa_decode does not take either)
bool plan_scores(ScoresPlan& sp, int B, int H, int K, int S_max, int d, int num_splits, bool paged, int sms) {
  if (!valid_decode_shape(B, H, K, S_max, d, paged) || num_splits < 0) return false;
  sp.pl = plan_decode(B, H, K, S_max, d, num_splits, GQA_BF16, sms, false, paged, true);
  if (sp.pl.ws_bytes == (size_t)-1) return false;
  const int G = H / K;
  const size_t parts = (size_t)B * K * sp.pl.nsplit * G;
  sp.ml_off = sp.pl.nsplit > 1 ? parts * d * sizeof(float) : 0;
  sp.queue_off = (sp.ml_off + parts * sizeof(float2) + 15) / 16 * 16;
  sp.x_off = sp.queue_off + 16;
  sp.bytes = sp.x_off + (size_t)B * H * (((size_t)S_max + 3) / 4 * 4) * sizeof(float);
  return true;
}

template <int D>
int launch_scores_decode(const ScoresPlan& sp, const DecodeParams& p, const gqa::ScoresParams& x, const void* kc,
                         const void* vc, uint64_t rows, cudaStream_t st) {
  CUtensorMap tk64, tv64, tk, tv;
  if (!encode_rows_bf16(&tk64, kc, rows, D, gqa::kDecTileKeys) ||
      !encode_rows_bf16(&tv64, vc, rows, D, gqa::kDecTileKeys) ||
      !encode_rows_bf16(&tk, kc, rows, D, gqa::kDecBoxRows) || !encode_rows_bf16(&tv, vc, rows, D, gqa::kDecBoxRows))
    return GQA_ERR_CUDA;
  using C = gqa::DecCfg<D>;
  static DeviceCache configured{};
  const int dev = current_device();
  if (dev >= 0 && dev < kMaxDevices && configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(gqa::decode_scores_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(gqa::decode_scores_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmemBytes) != cudaSuccess)
      return GQA_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  return gqa::launch_kernel(p.block_table ? gqa::decode_scores_kernel<D, true> : gqa::decode_scores_kernel<D, false>,
                            (unsigned)sp.pl.grid, gqa::kDecThreads, C::kSmemBytes, st, true, tk64, tv64, tk, tv, p, x);
}

int decode_scores_impl(void* out, float* scores, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* seqlens, int B, int H, int K, int S_max, int d, float scale, int num_splits,
                       void* workspace, size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream,
                       const PagedCache* pc) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_INVALID_ARG;
  if (num_splits < 0 || B < 0 || H <= 0 || K <= 0 || S_max <= 0) return GQA_ERR_INVALID_ARG;
  if (!valid_decode_shape(B, H, K, S_max, d, pc != nullptr)) return GQA_ERR_SHAPE;
  if (pc && !valid_paged(*pc, B, K)) return GQA_ERR_SHAPE;
  if (dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  if (B == 0) return GQA_OK;
  if (!out || !scores || !q || !k_cache || !v_cache || !seqlens || (pc && !pc->table)) return GQA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(scores) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return GQA_ERR_ALIGN;
  ScoresPlan sp;
  if (!plan_scores(sp, B, H, K, S_max, d, num_splits, pc != nullptr, sm_count(current_device()))) return GQA_ERR_SHAPE;
  if (!workspace || workspace_bytes < sp.bytes) return GQA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return GQA_ERR_ALIGN;
  // the join: four rows a thread, or eight where those CTAs would not all be resident (four per SM; both sides
  // measured beside scores_finish_kernel)
  const int acc_keys = 4 * gqa::kAccThreads;
  const bool eight = (long long)B * K * ((S_max + acc_keys - 1) / acc_keys) > 4ll * sm_count(current_device());
  const long long chunks = eight ? (S_max + 2 * acc_keys - 1) / (2 * acc_keys) : (S_max + acc_keys - 1) / acc_keys;
  if ((long long)B * K * chunks >= (1ll << 31)) return GQA_ERR_SHAPE;
  const DecodePlan& pl = sp.pl;
  char* ws = static_cast<char*>(workspace);
  DecodeParams p{};
  p.k_cache_w = const_cast<void*>(k_cache);  // the L2 warm-up's addresses; nothing is written
  p.v_cache_w = const_cast<void*>(v_cache);
  p.q = q;
  p.out = out;
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + sp.ml_off);
  p.ws_queue = reinterpret_cast<unsigned long long*>(ws + sp.queue_off);
  p.nitems = (int)((long long)B * K * pl.hslices * pl.nsplit);
  p.tag = next_call_tag();
  p.seqlens = seqlens;
  p.B = B;
  p.H = H;
  p.K = K;
  p.S_max = S_max;
  p.G = H / K;
  p.hslices = pl.hslices;
  p.chunk = pl.chunk;
  p.nsplit = pl.nsplit;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.block_table = pc ? pc->table : nullptr;
  p.max_blocks = pc ? pc->max_blocks : 0;
  p.block_size = pc ? pc->block_size : 0;
  p.num_blocks = pc ? pc->num_blocks : 0;
  gqa::ScoresParams x;
  x.x = reinterpret_cast<float*>(ws + sp.x_off);
  x.scores = scores;
  x.x_stride = (S_max + 3) / 4 * 4;
  cudaStream_t st = (cudaStream_t)stream;
  const uint64_t rows = pc ? (uint64_t)pc->num_blocks * K * pc->block_size : (uint64_t)B * K * S_max;
  int rc = d == 128 ? launch_scores_decode<128>(sp, p, x, k_cache, v_cache, rows, st)
                    : launch_scores_decode<64>(sp, p, x, k_cache, v_cache, rows, st);
  if (rc != GQA_OK) return rc;
  auto finish = [&](auto kernel) {
    return gqa::launch_kernel(kernel, (unsigned)(B * K * chunks), gqa::kAccThreads, 0, st, true, p, x, (int)chunks);
  };
  if (d == 128) return eight ? finish(gqa::scores_finish_kernel<128, 2>) : finish(gqa::scores_finish_kernel<128, 1>);
  return eight ? finish(gqa::scores_finish_kernel<64, 2>) : finish(gqa::scores_finish_kernel<64, 1>);
}

// ----------------------------------------------------------------------------
// gqa_kv_evict

struct EvictPlan {
  bool cta = false, fused = false;  // evict_cta_kernel; with the moves
  int seg_keys = 0, max_moves = 0;
  size_t done_off = 0, bytes = 0;
};

bool plan_evict(EvictPlan& pl, int B, int K, int S_max, int keep, int sms) {
  if (B < 0 || K <= 0 || S_max <= 0 || keep <= 0 || keep > S_max) return false;
  if ((long long)B * K * gqa::kEvCluster >= (1ll << 31)) return false;
  pl.max_moves = std::min(keep, S_max - keep);
  // a CTA per (b, g) while 8 rows a thread hold the cache (8 heads of 8192 rows: 18 us, as clusters 25); up to 16
  // where the clusters are more than the GPU holds at once (64 heads of 16384 rows: 32 us against 58; 8 of them: 35
  // against 21)
  pl.cta = S_max <= gqa::kEvCtaRows / 2 ||
           (S_max <= gqa::kEvCtaRows && (long long)B * K * gqa::kEvCluster > sms);
  pl.fused = pl.cta && pl.max_moves <= gqa::kEvFusedMoves;
  const int seg = ((S_max + gqa::kEvCluster - 1) / gqa::kEvCluster + 31) / 32 * 32;
  pl.seg_keys = std::min(seg, gqa::kEvMaxSegKeys);
  pl.done_off = pl.fused ? 0 : ((size_t)B * K * (1 + 4 * (size_t)pl.max_moves) * sizeof(int32_t) + 15) / 16 * 16;
  pl.bytes = pl.done_off + (pl.fused ? (size_t)std::max(B, 1) * sizeof(unsigned long long) : 0);
  return true;
}

template <bool kFused>
int launch_evict_cta(const gqa::EvictParams& p, cudaStream_t st) {
  auto run = [&](auto kernel) {
    return gqa::launch_kernel(kernel, (unsigned)(p.B * p.K), gqa::kEvThreads, 0, st, true, p);
  };
  if (p.S_max <= gqa::kEvThreads) return run(gqa::evict_cta_kernel<1, kFused>);
  if (p.S_max <= 2 * gqa::kEvThreads) return run(gqa::evict_cta_kernel<2, kFused>);
  if (p.S_max <= 4 * gqa::kEvThreads) return run(gqa::evict_cta_kernel<4, kFused>);
  if (p.S_max <= 8 * gqa::kEvThreads) return run(gqa::evict_cta_kernel<8, kFused>);
  return run(gqa::evict_cta_kernel<16, kFused>);
}

int kv_evict_impl(void* k_cache, void* v_cache, float* scores, int32_t* row_pos, int32_t* seqlens,
                  const int32_t* recent_from, int B, int K, int S_max, int d, int keep, int sinks, void* workspace,
                  size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream, const PagedCache* pc) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_INVALID_ARG;
  if (B < 0 || K <= 0 || S_max <= 0 || sinks < 0) return GQA_ERR_INVALID_ARG;
  if (keep <= 0 || keep > S_max || (d != 64 && d != 128)) return GQA_ERR_SHAPE;
  EvictPlan pl;
  if (!plan_evict(pl, B, K, S_max, keep, sm_count(current_device()))) return GQA_ERR_SHAPE;
  if (B == 0) return GQA_OK;
  if (!k_cache || !v_cache || !scores || !seqlens) return GQA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(scores)) return GQA_ERR_ALIGN;
  if (!workspace || workspace_bytes < pl.bytes) return GQA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return GQA_ERR_ALIGN;
  gqa::EvictParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.scores = scores;
  p.row_pos = row_pos;
  p.seqlens = seqlens;
  p.recent_from = recent_from;
  p.ws = static_cast<int32_t*>(workspace);
  p.done = reinterpret_cast<unsigned long long*>(static_cast<char*>(workspace) + pl.done_off);
  p.tag = next_call_tag();
  p.B = B;
  p.K = K;
  p.S_max = S_max;
  p.keep = keep;
  p.sinks = sinks;
  p.max_moves = pl.max_moves;
  p.seg_keys = pl.seg_keys;
  p.quads = S_max % 4 == 0 && aligned16(row_pos);
  p.row_chunks = d * (dtype == GQA_F32 ? 4 : 2) / 16;
  if (pc) {
    p.block_table = pc->table;
    p.num_blocks = pc->num_blocks;
    p.block_size = pc->block_size;
    p.max_blocks = pc->max_blocks;
  }
  const int dev = current_device();
  cudaStream_t st = (cudaStream_t)stream;
  const int units = B * K;
  int rc;
  if (pl.cta) {
    rc = pl.fused ? launch_evict_cta<true>(p, st) : launch_evict_cta<false>(p, st);
    if (rc != GQA_OK || pl.fused) return rc;
  } else {
    static DeviceCache configured{};
    if (dev >= 0 && dev < kMaxDevices && configured[dev].load(std::memory_order_acquire) == 0) {
      if (cudaFuncSetAttribute(gqa::evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               gqa::kEvStaticBytes + gqa::kEvMaxSegKeys * 4) != cudaSuccess)
        return GQA_ERR_CUDA;
      configured[dev].store(1, std::memory_order_release);
    }
    rc = gqa::launch_kernel(gqa::evict_select_kernel, (unsigned)(units * gqa::kEvCluster), gqa::kEvThreads,
                            (size_t)gqa::kEvStaticBytes + (size_t)pl.seg_keys * 4, st, true, p);
    if (rc != GQA_OK) return rc;
  }
  // as many CTAs as have rows to move, up to four per SM over all units
  const int per = gqa::kEvMoveThreads / (2 * p.row_chunks) * gqa::kEvFlight;  // rows a CTA has in flight
  p.ctas_per_unit =
      std::max(1, std::min((sm_count(dev) * 4 + units - 1) / units, (pl.max_moves + per - 1) / per));
  return gqa::launch_kernel(gqa::evict_move_kernel, (unsigned)(units * p.ctas_per_unit), gqa::kEvMoveThreads, 0, st,
                            true, p);
}

// One row of CTAs per sequence and tensor (grid y) for the 4-bit rows' kernels.
template <typename... KArgs, typename... Args>
int launch_mx_rows(void (*kernel)(KArgs...), int B, int T, int K, cudaStream_t st, Args... args) {
  const long long rows = (long long)T * K;
  if (rows >= (1ll << 31)) return GQA_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + gqa::kMxBlockRows - 1) / gqa::kMxBlockRows), std::min(2 * B, 65534));
  cfg.blockDim = dim3(gqa::kMxThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const QueryErrorScope scope;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return GQA_OK;
  scope.clear_own();
  return GQA_ERR_CUDA;
}

// ----------------------------------------------------------------------------
// gqa_prompt_scores

struct PromptPlan {
  int tile_tokens = 0, n_rt = 0, n_kt = 0;
  int key_splits = 1, row_splits = 1;  // of the kRows and the kKeys kernel
  size_t ml_off = 0, part_off = 0, queue_off = 0, bytes = 0;
};

bool plan_prompt(PromptPlan& pl, int B, int T, int H, int K, int S_max, int d, int sms) {
  if (T < 0 || !valid_decode_shape(B, H, K, S_max, d) || H / K > gqa::kPsRows) return false;
  if ((long long)B * T >= (1ll << 31)) return false;  // TMA coordinate
  pl.tile_tokens = gqa::kPsRows / (H / K);
  pl.n_rt = (T + pl.tile_tokens - 1) / pl.tile_tokens;
  pl.n_kt = (S_max + gqa::kPsRows - 1) / gqa::kPsRows;
  const long long units = (long long)B * K;
  // about two items (pairs of stationary tiles) per SM, four streamed tiles in each
  auto splits = [&](int tiles, int streamed) {
    const long long items = units * std::max((tiles + 1) / 2, 1);
    const long long want = (2ll * sms + items - 1) / std::max(items, 1ll);
    return (int)std::max(1ll, std::min<long long>(want, streamed / 4));
  };
  pl.key_splits = splits(pl.n_rt, pl.n_kt);
  pl.row_splits = splits(pl.n_kt, pl.n_rt);
  // below the work counter's range
  if (units * ((pl.n_rt + 1) / 2) * pl.key_splits + sms >= (1ll << gqa::kCntBits) ||
      units * ((pl.n_kt + 1) / 2) * pl.row_splits + sms >= (1ll << gqa::kCntBits))
    return false;
  const size_t rows = (size_t)units * pl.n_rt * gqa::kPsRows;
  pl.ml_off = rows * sizeof(float);
  pl.part_off = pl.ml_off + (pl.key_splits > 1 ? pl.key_splits * rows * sizeof(float2) : 0);
  const size_t part_bytes = pl.row_splits > 1 ? (size_t)pl.row_splits * units * S_max * sizeof(float) : 0;
  pl.queue_off = (pl.part_off + part_bytes + 15) / 16 * 16;
  pl.bytes = pl.queue_off + 32;  // a work counter for each of the two kernels
  return true;
}

// [tokens, H, D] bf16 as (64 columns, heads, tokens), box (64, box_heads, box_tokens), 128-byte swizzle: a tile's
// rows are its tokens' heads, one token after the other.
bool encode_head_rows_bf16(CUtensorMap* map, const void* base, uint64_t tokens, uint64_t H, uint64_t D,
                           uint32_t box_heads, uint32_t box_tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {D, H, tokens};
  cuuint64_t strides[2] = {D * 2, H * D * 2};
  cuuint32_t box[3] = {64, box_heads, box_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch_prompt(const PromptPlan& pl, gqa::PromptParams p, const void* q, const void* k_cache, cudaStream_t st) {
  CUtensorMap tq, tk;
  if (!encode_head_rows_bf16(&tq, q, (uint64_t)p.B * p.T, p.H, D, p.G, p.tile_tokens) ||
      !encode_rows_bf16(&tk, k_cache, (uint64_t)p.B * p.K * p.S_max, D, gqa::kPsRows))
    return GQA_ERR_CUDA;
  using C = gqa::PsCfg<D>;
  const auto rows_kernel = gqa::prompt_scores_kernel<D, gqa::kPsKindRows, false>;
  const auto keys_kernel = gqa::prompt_scores_kernel<D, gqa::kPsKindKeys, false>;
  const auto keys_zero_kernel = gqa::prompt_scores_kernel<D, gqa::kPsKindKeys, true>;
  static DeviceCache configured{};
  const int dev = current_device();
  if (dev >= 0 && dev < kMaxDevices && configured[dev].load(std::memory_order_acquire) == 0) {
    for (auto kernel : {rows_kernel, keys_kernel, keys_zero_kernel})
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
        return GQA_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  const int units = p.B * p.K;
  const int sms = sm_count(dev);
  p.splits = pl.key_splits;
  p.items = units * ((p.n_rt + 1) / 2) * p.splits;
  int rc = gqa::launch_kernel(rows_kernel, (unsigned)std::min(p.items, sms), gqa::kPsThreads, C::kSmemBytes, st, true,
                              tq, tk, p);
  if (rc != GQA_OK) return rc;
  if (p.splits > 1) {
    const long long rows = (long long)units * p.n_rt * gqa::kPsRows;
    rc = gqa::launch_kernel(gqa::prompt_lse_kernel, (unsigned)grid_for(rows, 256, sms), 256, 0, st, true, p.nlse,
                            (const float2*)p.ml, rows, p.splits);
    if (rc != GQA_OK) return rc;
  }
  p.splits = pl.row_splits;
  p.items = units * ((p.n_kt + 1) / 2) * p.splits;
  p.queue += 2;
  rc = gqa::launch_kernel(p.tile_tokens * p.G == gqa::kPsRows ? keys_kernel : keys_zero_kernel,
                          (unsigned)std::min(p.items, sms), gqa::kPsThreads, C::kSmemBytes, st, true, tq, tk, p);
  if (rc != GQA_OK || p.splits == 1) return rc;
  return gqa::launch_kernel(gqa::prompt_add_kernel, (unsigned)grid_for((long long)units * p.S_max, 256, sms), 256, 0,
                            st, true, p.scores, (const float*)p.part, p.seqlens, units, p.K, p.S_max, p.splits);
}

// ----------------------------------------------------------------------------
// gqa_decode_mxfp4

// [rows, 64] bytes of codes (rows even) as [rows / 2, 128], 128-byte swizzle, box of box_rows rows
bool encode_rows_mx(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  return encode_rows_u8(map, base, rows / 2, box_rows / 2);
}

struct MxPlan {
  int hslices = 1, chunk = 0, nsplit = 1, grid = 1;
  size_t ml_off = 0, queue_off = 0, bytes = 0;
};

bool plan_mx(MxPlan& pl, int B, int H, int K, int S_max, int d, int num_splits, int sms) {
  if (!valid_decode_shape(B, H, K, S_max, d) || d != gqa::kMxD || S_max % 4 != 0 || num_splits < 0) return false;
  const int G = H / K;
  pl.hslices = (G + gqa::kDecHeadsPerCta - 1) / gqa::kDecHeadsPerCta;
  const long long units = (long long)B * K * pl.hslices;
  const int max_splits = std::min((S_max + gqa::kMxTileKeys - 1) / gqa::kMxTileKeys, gqa::kMaxCombineSplits);
  int splits;
  if (num_splits > 0) {
    splits = std::min(num_splits, max_splits);
  } else {
    // Items per resident CTA: sequences of one length want few, unequal ones many, and the plan does not know the
    // lengths. 8 KV heads of 4 query heads, 16384 tokens each / 1K to 16K, us at one, two, four and six:
    //    16 units   15.8  17.8  17.8  17.9 /  14.7  13.1  13.1  13.1
    //    64         38.0  39.0  43.3  43.5 /  35.0  27.6  30.6  30.8
    //    96         59.7  58.0  57.4  58.5 /  46.0  39.2  41.6  42.6
    //   128         73.1  72.7  67.2  73.0 /  54.6  49.9  50.7  50.9
    //   192         94.6  93.8  98.7  94.4 /  70.7  68.3  62.6  62.5
    //   256        138.6 117.6 123.9 124.5 /  97.8  85.4  81.2  80.9
    //   512        260   221   237   227   / 178   148   137   133
    // Two is the best or near it for both below 128 units; from there on two costs unequal lengths up to 9 % and
    // four equal ones up to 7 %, and a batch of many sequences is seldom of one length.
    const long long target = (units >= 128 ? 4ll : 2ll) * gqa::kMxCtasPerSm * sms;
    splits = (int)std::max<long long>(1, (target + units - 1) / std::max<long long>(units, 1));
    splits = std::min(splits, std::max(1, (S_max + 511) / 512));
    splits = std::min(splits, max_splits);
  }
  const int chunk = (S_max + splits - 1) / splits;
  pl.chunk = (chunk + gqa::kMxTileKeys - 1) / gqa::kMxTileKeys * gqa::kMxTileKeys;
  pl.nsplit = (S_max + pl.chunk - 1) / pl.chunk;
  const long long items = units * pl.nsplit;
  pl.grid = (int)std::max<long long>(1, std::min<long long>(items, (long long)gqa::kMxCtasPerSm * sms));
  if (items + pl.grid >= (1ll << gqa::kCntBits)) return false;  // beyond the work counter
  const size_t parts = pl.nsplit > 1 ? (size_t)B * K * pl.nsplit * G : 0;
  pl.ml_off = parts * d * sizeof(float);
  pl.queue_off = (pl.ml_off + parts * sizeof(float2) + 15) / 16 * 16;
  pl.bytes = pl.queue_off + 16;
  return true;
}

}  // namespace

extern "C" {

int gqa_rope_table(float* rope, int max_pos, int rotary_dim, double theta, gqa_stream_t stream) {
  if (max_pos < 0 || !(theta > 0.0)) return GQA_ERR_INVALID_ARG;
  if (rotary_dim <= 0 || rotary_dim % 2 != 0) return GQA_ERR_SHAPE;
  if (max_pos == 0) return GQA_OK;
  if (!rope) return GQA_ERR_INVALID_ARG;
  if (!aligned16(rope)) return GQA_ERR_ALIGN;
  const int grid = grid_for((long long)max_pos * (rotary_dim / 2), 256, sm_count(current_device()));
  return gqa::launch_kernel(gqa::rope_table_kernel, (unsigned)grid, 256, 0, (cudaStream_t)stream, false, rope, max_pos,
                            rotary_dim / 2, theta);
}

int gqa_qk_norm_rope(void* q_out, void* k_out, void* k_cache, void* v_cache, int32_t* row_pos, const void* q,
                     const void* k, const void* v, const void* q_weight, const void* k_weight, const float* rope,
                     const int32_t* positions, const int32_t* rows, int B, int T, int H, int K, int S_max, int d,
                     int64_t q_stride, int64_t k_stride, int64_t v_stride, int rotary_dim, int max_pos,
                     int interleaved, float eps, gqa_dtype dtype, gqa_stream_t stream) {
  return norm_rope_impl(q_out, k_out, k_cache, v_cache, row_pos, q, k, v, q_weight, k_weight, rope, positions, rows, B,
                        T, H, K, S_max, d, q_stride, k_stride, v_stride, rotary_dim, max_pos, interleaved, eps, dtype,
                        stream, nullptr);
}

int gqa_qk_norm_rope_paged(void* q_out, void* k_out, void* k_pool, void* v_pool, int32_t* row_pos, const void* q,
                           const void* k, const void* v, const void* q_weight, const void* k_weight, const float* rope,
                           const int32_t* positions, const int32_t* block_table, const int32_t* rows, int B, int T,
                           int H, int K, int d, int num_blocks, int block_size, int max_blocks, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, int rotary_dim, int max_pos, int interleaved, float eps,
                           gqa_dtype dtype, gqa_stream_t stream) {
  if (B < 0 || K <= 0) return GQA_ERR_INVALID_ARG;
  const PagedCache pc = paged_cache(block_table, num_blocks, block_size, max_blocks);
  if (!valid_paged(pc, B, K)) return GQA_ERR_SHAPE;
  if (B > 0 && T != 0 && (!block_table || !k_pool || !v_pool)) return GQA_ERR_INVALID_ARG;
  return norm_rope_impl(q_out, k_out, k_pool, v_pool, row_pos, q, k, v, q_weight, k_weight, rope, positions, rows, B,
                        T, H, K, max_blocks * block_size, d, q_stride, k_stride, v_stride, rotary_dim, max_pos,
                        interleaved, eps, dtype, stream, &pc);
}

size_t gqa_decode_scores_workspace_bytes(int B, int H, int K, int S_max, int d, int num_splits) {
  return most_over_batches(B, [&](int b, int sms) {
    ScoresPlan sp;
    return plan_scores(sp, b, H, K, S_max, d, num_splits, false, sms) ? sp.bytes : 0;
  });
}

size_t gqa_decode_scores_paged_workspace_bytes(int B, int H, int K, int d, int block_size, int max_blocks,
                                               int num_splits) {
  if (block_size <= 0 || block_size % 16 != 0 || max_blocks <= 0 || (long long)max_blocks * block_size >= (1ll << 31))
    return 0;
  return most_over_batches(B, [&](int b, int sms) {
    ScoresPlan sp;
    return plan_scores(sp, b, H, K, max_blocks * block_size, d, num_splits, true, sms) ? sp.bytes : 0;
  });
}

int gqa_decode_scores(void* out, float* scores, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* seqlens, int B, int H, int K, int S_max, int d, float scale, int num_splits,
                      void* workspace, size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream) {
  return decode_scores_impl(out, scores, q, k_cache, v_cache, seqlens, B, H, K, S_max, d, scale, num_splits, workspace,
                            workspace_bytes, dtype, stream, nullptr);
}

int gqa_decode_scores_paged(void* out, float* scores, const void* q, const void* k_pool, const void* v_pool,
                            const int32_t* block_table, const int32_t* seqlens, int B, int H, int K, int d,
                            int num_blocks, int block_size, int max_blocks, float scale, int num_splits,
                            void* workspace, size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream) {
  if (block_size <= 0 || max_blocks <= 0 || (long long)max_blocks * block_size >= (1ll << 31)) return GQA_ERR_SHAPE;
  const PagedCache pc = paged_cache(block_table, num_blocks, block_size, max_blocks);
  return decode_scores_impl(out, scores, q, k_pool, v_pool, seqlens, B, H, K, max_blocks * block_size, d, scale,
                            num_splits, workspace, workspace_bytes, dtype, stream, &pc);
}

size_t gqa_kv_evict_workspace_bytes(int B, int K, int S_max, int keep) {
  return most_over_batches(B, [&](int b, int sms) {
    EvictPlan pl;
    return plan_evict(pl, b, K, S_max, keep, sms) ? pl.bytes : 0;
  });
}

int gqa_kv_evict(void* k_cache, void* v_cache, float* scores, int32_t* row_pos, int32_t* seqlens,
                 const int32_t* recent_from, int B, int K, int S_max, int d, int keep, int sinks, void* workspace,
                 size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream) {
  return kv_evict_impl(k_cache, v_cache, scores, row_pos, seqlens, recent_from, B, K, S_max, d, keep, sinks, workspace,
                       workspace_bytes, dtype, stream, nullptr);
}

int gqa_kv_evict_paged(void* k_pool, void* v_pool, const int32_t* block_table, float* scores, int32_t* row_pos,
                       int32_t* seqlens, const int32_t* recent_from, int B, int K, int d, int num_blocks,
                       int block_size, int max_blocks, int keep, int sinks, void* workspace, size_t workspace_bytes,
                       gqa_dtype dtype, gqa_stream_t stream) {
  if (B < 0 || K <= 0) return GQA_ERR_INVALID_ARG;
  const PagedCache pc = paged_cache(block_table, num_blocks, block_size, max_blocks);
  if (!valid_paged(pc, B, K)) return GQA_ERR_SHAPE;
  if (B > 0 && !block_table) return GQA_ERR_INVALID_ARG;
  return kv_evict_impl(k_pool, v_pool, scores, row_pos, seqlens, recent_from, B, K, max_blocks * block_size, d, keep,
                       sinks, workspace, workspace_bytes, dtype, stream, &pc);
}

int gqa_kv_append_mxfp4(uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, const void* k_new,
                        const void* v_new, const int32_t* pos, int B, int T, int K, int S_max, int d,
                        gqa_stream_t stream) {
  if (B < 0 || T < 0 || K <= 0 || S_max <= 0) return GQA_ERR_INVALID_ARG;
  if (d != gqa::kMxD) return GQA_ERR_UNSUPPORTED;
  if (S_max % 4 != 0 || T > S_max) return GQA_ERR_SHAPE;
  if (B == 0 || T == 0) return GQA_OK;
  if (!k_codes || !k_scales || !v_codes || !v_scales || !k_new || !v_new || !pos) return GQA_ERR_INVALID_ARG;
  if (!aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales) ||
      !aligned16(k_new) || !aligned16(v_new))
    return GQA_ERR_ALIGN;
  return launch_mx_rows(gqa::kv_append_mxfp4_kernel, B, T, K, (cudaStream_t)stream, k_codes, k_scales, v_codes,
                        v_scales, static_cast<const uint8_t*>(k_new), static_cast<const uint8_t*>(v_new), pos, B, T, K,
                        S_max);
}

int gqa_kv_read_mxfp4(void* k_out, void* v_out, const uint8_t* k_codes, const uint8_t* k_scales,
                      const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* pos, int B, int T, int K,
                      int S_max, int d, gqa_stream_t stream) {
  if (B < 0 || T < 0 || K <= 0 || S_max <= 0) return GQA_ERR_INVALID_ARG;
  if (d != gqa::kMxD) return GQA_ERR_UNSUPPORTED;
  if (S_max % 4 != 0 || T > S_max) return GQA_ERR_SHAPE;
  if (B == 0 || T == 0) return GQA_OK;
  if (!k_codes || !k_scales || !v_codes || !v_scales || !k_out || !v_out || !pos) return GQA_ERR_INVALID_ARG;
  if (!aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales) ||
      !aligned16(k_out) || !aligned16(v_out))
    return GQA_ERR_ALIGN;
  return launch_mx_rows(gqa::kv_read_mxfp4_kernel, B, T, K, (cudaStream_t)stream, static_cast<uint8_t*>(k_out),
                        static_cast<uint8_t*>(v_out), k_codes, k_scales, v_codes, v_scales, pos, B, T, K, S_max);
}

size_t gqa_prompt_scores_workspace_bytes(int B, int T, int H, int K, int S_max, int d) {
  return most_over_batches(B, [&](int b, int sms) {
    PromptPlan pl;
    return plan_prompt(pl, b, T, H, K, S_max, d, sms) ? pl.bytes : 0;
  });
}

int gqa_prompt_scores(float* scores, const void* q, const void* k_cache, const int32_t* seqlens, int B, int T, int H,
                      int K, int S_max, int d, float scale, void* workspace, size_t workspace_bytes, gqa_dtype dtype,
                      gqa_stream_t stream) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || H <= 0 || K <= 0 || S_max <= 0) return GQA_ERR_INVALID_ARG;
  PromptPlan pl;
  if (!plan_prompt(pl, B, T, H, K, S_max, d, sm_count(current_device()))) return GQA_ERR_SHAPE;
  if (dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return GQA_OK;
  if (!scores || !q || !k_cache || !seqlens) return GQA_ERR_INVALID_ARG;
  if (!aligned16(scores) || !aligned16(q) || !aligned16(k_cache)) return GQA_ERR_ALIGN;
  if (!workspace || workspace_bytes < pl.bytes) return GQA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return GQA_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  gqa::PromptParams p{};
  p.scores = scores;
  p.nlse = reinterpret_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + pl.ml_off);
  p.part = reinterpret_cast<float*>(ws + pl.part_off);
  p.queue = reinterpret_cast<unsigned long long*>(ws + pl.queue_off);
  p.tag = next_call_tag();
  p.seqlens = seqlens;
  p.B = B;
  p.T = T;
  p.H = H;
  p.K = K;
  p.G = H / K;
  p.S_max = S_max;
  p.tile_tokens = pl.tile_tokens;
  p.n_rt = pl.n_rt;
  p.n_kt = pl.n_kt;
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = (cudaStream_t)stream;
  return d == 128 ? launch_prompt<128>(pl, p, q, k_cache, st) : launch_prompt<64>(pl, p, q, k_cache, st);
}

size_t gqa_decode_mxfp4_workspace_bytes(int B, int H, int K, int S_max, int d, int num_splits) {
  return most_over_batches(B, [&](int b, int sms) {
    MxPlan pl;
    return plan_mx(pl, b, H, K, S_max, d, num_splits, sms) ? pl.bytes : 0;
  });
}

int gqa_decode_mxfp4(void* out, const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                     const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* seqlens, int B, int H, int K,
                     int S_max, int d, float scale, int num_splits, void* workspace, size_t workspace_bytes,
                     gqa_stream_t stream) {
  if (num_splits < 0 || B < 0 || H <= 0 || K <= 0 || S_max <= 0) return GQA_ERR_INVALID_ARG;
  if (d != gqa::kMxD) return GQA_ERR_UNSUPPORTED;
  const int dev = current_device();
  const int sms = sm_count(dev);
  MxPlan pl;
  if (!plan_mx(pl, B, H, K, S_max, d, num_splits, sms)) return GQA_ERR_SHAPE;
  if (B == 0) return GQA_OK;
  if (!out || !q || !k_codes || !k_scales || !v_codes || !v_scales || !seqlens) return GQA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) ||
      !aligned16(v_scales))
    return GQA_ERR_ALIGN;
  if (!workspace || workspace_bytes < pl.bytes) return GQA_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return GQA_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  DecodeParams p{};
  p.k_cache_w = const_cast<uint8_t*>(k_codes);  // the L2 warm-up's addresses; nothing is written
  p.v_cache_w = const_cast<uint8_t*>(v_codes);
  p.q = q;
  p.out = out;
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + pl.ml_off);
  p.ws_queue = reinterpret_cast<unsigned long long*>(ws + pl.queue_off);
  p.nitems = (int)((long long)B * K * pl.hslices * pl.nsplit);
  p.tag = next_call_tag();
  p.seqlens = seqlens;
  p.B = B;
  p.H = H;
  p.K = K;
  p.S_max = S_max;
  p.G = H / K;
  p.hslices = pl.hslices;
  p.chunk = pl.chunk;
  p.nsplit = pl.nsplit;
  p.scale_log2 = scale * 1.4426950408889634f;
  const gqa::MxParams mp{k_scales, v_scales};
  const uint64_t rows = (uint64_t)B * K * S_max;
  CUtensorMap tk, tv, tk16, tv16;
  if (!encode_rows_mx(&tk, k_codes, rows, gqa::kMxTileKeys) || !encode_rows_mx(&tv, v_codes, rows, gqa::kMxTileKeys) ||
      !encode_rows_mx(&tk16, k_codes, rows, gqa::kDecBoxRows) ||
      !encode_rows_mx(&tv16, v_codes, rows, gqa::kDecBoxRows))
    return GQA_ERR_CUDA;
  static DeviceCache configured{};
  if (dev >= 0 && dev < kMaxDevices && configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(gqa::decode_mxfp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gqa::MxCfg::kSmemBytes) != cudaSuccess)
      return GQA_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = gqa::launch_kernel(gqa::decode_mxfp4_kernel, (unsigned)pl.grid, gqa::kMxDecThreads,
                                    gqa::MxCfg::kSmemBytes, st, true, tk, tv, tk16, tv16, p, mp);
  if (rc != GQA_OK || pl.nsplit == 1) return rc;
  return launch_combine(out, p, seqlens, H, K, S_max, p.G, pl.chunk, pl.nsplit, 1, d, GQA_BF16, pl.nsplit > 32,
                        (long long)B * H, st);
}

}  // extern "C"
