// gqa_decode_mxfp4: the decode of decode.cuh over the 4-bit cache of mxfp4.cuh.
//
// Same work items, ring and split merge. A stage holds 128 keys: K and V
// codes (64-byte rows), their scales (a 32-bit word per key
// and tensor) and, with an item's first tile, its q rows. Each of the four
// consumer warps takes 32 keys, as two independent 16-key blocks.
//
// Codes become fp16 by the hardware's e2m1 conversion, two at a time, and go
// into fp16 MMAs with fp32 sums; the scales stay out of the products:
//   S = sum over 32-dim blocks of 2^(E_k - 127) (q . code): an ldmatrix gives
//     a lane 8 codes of one block of its key, so two 16-dim MMAs cover a block
//     (q in the same order of dims), and their sum is scaled in fp32. q is
//     held in fp16 over a power of two of its own per head, 2^8 at the top:
//     exact for elements down to 2^-25 of the head's largest.
//   O = sum over keys of P (V codes) 2^(E_v - 127): the scale goes with P.
//     A transposing ldmatrix gives a lane 4 dims of keys 2 t and 2 t + 1, and
//     a second one of 2 t + 8 and 2 t + 9; interleaving the two words' nibbles
//     makes each byte one dim of two keys (8 apart), which the conversion
//     turns into a register of the A operand. P^T takes the same key order.
//
// P 2^(E_v - 127) leaves fp16's range, so each warp holds a reference exponent
// R per block and multiplies 2^13 P by 2^(E_v - R + 1). At E_v = R - j that
// product holds P's 11 bits down to P = 2^(j - 28) and multiples of 2^(j - 38)
// below. It is taken while every E_v of the step lies in [R - 11, R], so that a
// weight is off by 2^-12 of itself or 2^-28 of the largest at most: the
// rounding of half a million equal weights stays below bf16's. (With 2^10 P and
// j up to 15, 60000 weights of 1.06 2^-17 beside one of 1 were off by 6 %
// each.) A step outside the range raises R, or, where its own scales lie
// further apart, takes the same product in bf16 (2^-9 of each weight; a further
// conversion per code: 138 us for the 32 sequences below where every step does,
// 84 with the same random rows and scales within 2^9). There R need not reach
// every E_v, only the largest P 2^(E_v - 127): a value of a huge scale and no
// weight leaves the others theirs. What lies 2^126 below the largest product of
// a block counts as zero.
//
// P is relative to a reference score m that follows the running maximum only
// when a step exceeds it by 2^1: the exchange between lanes that finds the
// maximum is then a rare step, and P stays at 2 or below. A lag of 2^4 would
// cost three bits of P for 1 to 2 % of the time (the batches below: 27.1 and
// 73.0 us against 27.4 and 74.5 at the same time).
//
// Bound: the consumers. 136 bytes a key would stream at 5.6 TB/s through this
// ring (47 us for 32 sequences of 1K to 16K tokens, 64 query and 8 KV heads);
// with both products it is 75 us (3.5 TB/s): 501 instructions for 32 keys of 8
// heads, half of them on the half-rate ALU pipe (codes, nibbles, scales). At a
// lag of 2^4 (480 instructions, 72 us) the scores alone took 54 us, the weighted
// sum alone 60. 8 x 8192 tokens of 32 and 8 heads, with the append before it: 27
// us. No faster: eight consumer warps a CTA (76 us for 72), a ring of four
// stages (72 to 74), V codes loaded before the softmax, L2 prefetches.
#pragma once

#include "decode.cuh"
#include "mxfp4.cuh"

namespace gqa {

constexpr int kMxWarps = 4;  // consumers
constexpr int kMxDecThreads = (kMxWarps + 1) * 32;
constexpr int kMxWarpKeys = 32;
constexpr int kMxTileKeys = kMxWarps * kMxWarpKeys;
constexpr int kMxStages = 3;
constexpr int kMxCtasPerSm = 3;
constexpr float kMxLag = 1.f;    // how far scores may pass m
constexpr float kMxBias = 13.f;  // 2^(x - m + kMxBias + 1) stays below fp16's 65504
constexpr int kMxSpan = 11;      // E_v of the fp16 product: [R - kMxSpan, R]
constexpr int kMxHeadroom = 2;   // a raised R lies this far above the step's largest E_v
constexpr int kMxSmall = 8;      // keys of weight 2^-8 or more raise R to their E_v

struct MxCfg {
  static constexpr int kCodeBytes = kMxTileKeys * kMxRowBytes;
  static constexpr int kScaleOff = 2 * kCodeBytes;                  // K scales, then V scales
  static constexpr int kQOff = kScaleOff + 2 * kMxTileKeys * 4;
  static constexpr int kStageBytes = kQOff + kDecHeadsPerCta * kMxD * 2;
  static constexpr int kMergeFloats = kMxWarps * (2 * kDecHeadsPerCta + kDecHeadsPerCta * kMxD);
  static constexpr int kMergeOff = kMxStages * kStageBytes;
  static constexpr int kInfoOff = kMergeOff + kMergeFloats * 4;
  static constexpr int kBarOff = kInfoOff + kMxStages * 16;
  static constexpr int kSmemBytes = kBarOff + 2 * kMxStages * 8;
};
static_assert(MxCfg::kStageBytes % 1024 == 0, "stages start on the swizzle pattern");
static_assert(kMxSpan <= 15, "a half's exponent field holds E - R + 16 in five bits");

struct MxParams {
  const uint8_t *k_scales, *v_scales;
};

// Byte offset of 16-byte chunk `chunk` (0..3) of key `key` of a tile of codes:
// TMA writes two keys as one 128-byte row, 128-byte swizzled (64-byte rows
// would be twice as many rows for TMA; eight consecutive keys' chunks lie in
// eight different bank groups either way).
__device__ __forceinline__ uint32_t mx_at(uint32_t key, uint32_t chunk) {
  return sw128(key >> 1, (key & 1u) * 4u + chunk);
}

// Four scale bytes -> their values 2^(E - 127) (NaN for 255), by way of bf16, which holds every one of them.
__device__ __forceinline__ void e8m0x4_to_f32(uint32_t w, float (&s)[4]) {
  uint32_t lo, hi;
  asm("{\n .reg .b16 h0, h1;\n mov.b32 {h0, h1}, %2;\n"
      " cvt.rn.bf16x2.ue8m0x2 %0, h0;\n cvt.rn.bf16x2.ue8m0x2 %1, h1;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  s[0] = __uint_as_float(lo << 16);
  s[1] = __uint_as_float(lo & 0xffff0000u);
  s[2] = __uint_as_float(hi << 16);
  s[3] = __uint_as_float(hi & 0xffff0000u);
}

// D(16x8) = A(16x16) * B(16x8), fp16 operands
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t c;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(c) : "r"(a), "r"(b), "r"(sel));
  return c;
}

// The low (even) and the high (odd) nibbles of a's and b's bytes, a's in the low halves
__device__ __forceinline__ uint32_t even_nibbles(uint32_t a, uint32_t b) {
  return (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
}
__device__ __forceinline__ uint32_t odd_nibbles(uint32_t a, uint32_t b) {
  return ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
}

// Running state of one consumer warp. l is held times 2^kMxBias, o times twice
// that and over 2^(R - 127) of its 32-dim block; m is the scores' reference.
struct MxState {
  float m_a, m_b, l_a, l_b;
  uint32_t ref;  // R of block i in byte i, 16 or more (above kMxBias + 1); the same in all lanes
  float o[kMxD / 16][4];
  __device__ __forceinline__ void reset() {
    m_a = m_b = -INFINITY;
    l_a = l_b = 0.f;
    ref = 0x10101010u;
#pragma unroll
    for (int i = 0; i < kMxD / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }
};

// Q^T as the fp16 B operand: in the MMA ks = 2 b + s the lane holds head
// lane / 4, dims 32 b + 8 (lane % 4) + 4 s + {0, 1} and + {2, 3}. Returns the
// power of two that the head's elements were divided by.
__device__ __forceinline__ float load_q_frag_mx(uint32_t (&qf)[kMxD / 16][2], const __nv_bfloat16* q, int lane,
                                                int nh) {
  const int hn = lane >> 2;
  const bool hv = hn < nh;
  const uint4* row = reinterpret_cast<const uint4*>(q + (size_t)(hv ? hn : 0) * kMxD);
  uint32_t u[4][4];
  uint32_t top = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint4 w = row[b * 4 + (lane & 3)];
    u[b][0] = w.x, u[b][1] = w.y, u[b][2] = w.z, u[b][3] = w.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max((u[b][i] << 16) & 0x7fff0000u, u[b][i] & 0x7fff0000u));
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 2^8 / 2^floor(log2 top): exponent fields 27 .. 253 keep both powers in range (an element of 254 is below 2^10 then)
  const uint32_t e = min(max(top >> 23, 27u), 253u);
  const float down = __uint_as_float((262u - e) << 23), up = __uint_as_float((e - 8u) << 23);
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(u[b][i] << 16) * down, hi = __uint_as_float(u[b][i] & 0xffff0000u) * down;
      qf[2 * b + (i >> 1)][i & 1] = hv ? pack_f16x2(lo, hi) : 0u;
    }
  return up;
}

// The references to `ref`, each at or above what it was
__device__ __forceinline__ void mx_raise(MxState& st, uint32_t ref) {
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t up = ((ref >> (8 * b)) & 255u) - ((st.ref >> (8 * b)) & 255u);
    const float f = up > 126u ? 0.f : __uint_as_float((127u - up) << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[2 * b + i][j] *= f;
  }
  st.ref = ref;
}

// The step's V scales do not lie within every block's [R - kMxSpan, R] (in some
// lane). Where each block's are close enough to one another for the fp16
// product, raise the references that have to be. True if all lie within then.
__device__ __forceinline__ bool mx_rebase(MxState& st, uint32_t own, bool valid) {
  uint32_t ref = 0;
  bool fits = true;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t e = (own >> (8 * b)) & 255u;
    const uint32_t top = __reduce_max_sync(0xffffffffu, valid ? e : 0u);
    const uint32_t low = __reduce_min_sync(0xffffffffu, valid ? e : 255u);
    const uint32_t r = max((st.ref >> (8 * b)) & 255u, min(min(top + kMxHeadroom, low + kMxSpan), 254u));
    fits = fits && top <= r && r <= low + kMxSpan;  // a NaN's 255 does not
    ref |= r << (8 * b);
  }
  if (fits) mx_raise(st, ref);
  return fits;
}

// For the bfloat16 product, where some E_v lies above its R: R at floor(log2 P)
// + E_v of every key and head or above, so that no product overflows, and at the
// E_v of keys of weight 2^-kMxSmall or more, so that there is seldom a next time.
// No higher, so that values of a large scale and no weight do not push the
// others out of float32's range.
__device__ __forceinline__ void mx_follow(MxState& st, const float (&pa)[4], const float (&pb)[4], const uint32_t* sv,
                                          int key0, int rows, int head, int nh) {
  int need[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float p = fmaxf(head < nh ? pa[i] : 0.f, head + 1 < nh ? pb[i] : 0.f);
    const int lg = (int)(__float_as_uint(p) >> 23) - 127 - (int)kMxBias;
    if (key0 + 8 * i >= rows || lg < -126) continue;
    const uint32_t e = sv[key0 + 8 * i];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int eb = (int)((e >> (8 * b)) & 255u);
      if (eb != 255) need[b] = max(need[b], eb + min(lg + kMxSmall, 0));
    }
  }
  uint32_t ref = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    ref |= max((st.ref >> (8 * b)) & 255u, min((uint32_t)__reduce_max_sync(0xffffffffu, need[b]), 254u)) << (8 * b);
  mx_raise(st, ref);
}

// 2^(E - R + 1) as bf16 bits (NaN for E = 255). Beyond 2^127 P is below 2^-126 of the largest: 0, as below 2^-126.
__device__ __forceinline__ uint32_t mx_bf16_scale(uint32_t e, uint32_t r) {
  const uint32_t f = e + 128u - r;  // exponent field
  return e == 255u ? 0x7fc0u : f - 1u < 254u ? f << 7 : 0u;
}

// One warp's 32 keys (kb .. kb + 31) of the tile in `stage`; `rows` keys of
// the tile are valid, kb < rows; nh heads. f_a, f_b: scale * log2(e) * the power
// of two of the lane's heads.
__device__ __forceinline__ void warp_tile_mx(MxState& st, const uint32_t (&qf)[kMxD / 16][2], float f_a, float f_b,
                                             const uint8_t* stage, int kb, int rows, int lane, int nh) {
  using C = MxCfg;
  const uint32_t k_base = smem_u32(stage);
  const uint32_t v_base = k_base + C::kCodeBytes;
  const uint32_t* sk = reinterpret_cast<const uint32_t*>(stage + C::kScaleOff);
  const uint32_t* sv = sk + kMxTileKeys;
  // ldmatrix: (rows 0-7, chunk c) (rows 8-15, chunk c) (rows 0-7, chunk c + 1) (rows 8-15, chunk c + 1)
  const int row = kb + (lane & 7) + ((lane >> 3) & 1) * 8;
  const int ch = lane >> 4;

  // scores: key kb + lane / 4 + 8 i, i < 4
  const int key0 = kb + (lane >> 2);
  float xa[4], xb[4];
#pragma unroll
  for (int nb = 0; nb < 2; ++nb) {
    float s0[4], s1[4];
    e8m0x4_to_f32(sk[key0 + 16 * nb], s0);
    e8m0x4_to_f32(sk[key0 + 16 * nb + 8], s1);
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t r[4];
      ldmatrix_x4(k_base + mx_at(row + 16 * nb, 2 * j + ch), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = 2 * j + i;
        uint32_t lo[4], hi[4];
        e2m1x8_to_f16(r[2 * i], lo);
        e2m1x8_to_f16(r[2 * i + 1], hi);
        float c[4];
        mma_f16_16816_zero(c, lo[0], hi[0], lo[1], hi[1], qf[2 * b][0], qf[2 * b][1]);
        mma_f16_16816(c, lo[2], hi[2], lo[3], hi[3], qf[2 * b + 1][0], qf[2 * b + 1][1]);
        t[0] = fmaf(c[0], s0[b], t[0]);
        t[1] = fmaf(c[1], s0[b], t[1]);
        t[2] = fmaf(c[2], s1[b], t[2]);
        t[3] = fmaf(c[3], s1[b], t[3]);
      }
    }
    xa[2 * nb] = t[0] * f_a;
    xb[2 * nb] = t[1] * f_b;
    xa[2 * nb + 1] = t[2] * f_a;
    xb[2 * nb + 1] = t[3] * f_b;
  }
  const bool partial = kb + kMxWarpKeys > rows;
  if (partial) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (key0 + 8 * i >= rows) xa[i] = xb[i] = -INFINITY;
  }

  float mx_a = fmaxf(fmaxf(xa[0], xa[1]), fmaxf(xa[2], xa[3]));
  float mx_b = fmaxf(fmaxf(xb[0], xb[1]), fmaxf(xb[2], xb[3]));
  if (__any_sync(0xffffffffu, mx_a > st.m_a + kMxLag || mx_b > st.m_b + kMxLag)) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
    }
    const float mn_a = fmaxf(st.m_a, mx_a), mn_b = fmaxf(st.m_b, mx_b);
    // scores below float32's range alone so far: they weigh nothing, against any finite reference
    const float al_a = fast_exp2(st.m_a - (mn_a == -INFINITY ? 0.f : mn_a));
    const float al_b = fast_exp2(st.m_b - (mn_b == -INFINITY ? 0.f : mn_b));
    st.m_a = mn_a;
    st.m_b = mn_b;
    st.l_a *= al_a;
    st.l_b *= al_b;
#pragma unroll
    for (int md = 0; md < kMxD / 16; ++md) {
      st.o[md][0] *= al_a;
      st.o[md][1] *= al_b;
      st.o[md][2] *= al_a;
      st.o[md][3] *= al_b;
    }
  }
  float pa[4], pb[4];
  const float r_a = (st.m_a == -INFINITY ? 0.f : st.m_a) - kMxBias;
  const float r_b = (st.m_b == -INFINITY ? 0.f : st.m_b) - kMxBias;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pa[i] = fast_exp2(xa[i] - r_a);
    pb[i] = fast_exp2(xb[i] - r_b);
  }
  st.l_a += (pa[0] + pa[1]) + (pa[2] + pa[3]);
  st.l_b += (pb[0] + pb[1]) + (pb[2] + pb[3]);

  // V scales: the keys 2 (lane % 4) + {0, 1} + 8 i of the P^T operand; those past the valid rows: 2^0 times P = 0
  uint2 ev[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ev[i] = *reinterpret_cast<const uint2*>(sv + kb + 2 * (lane & 3) + 8 * i);
  const uint32_t own = sv[kb + lane];
  const bool own_valid = kb + lane < rows;
  // R - E of each byte in 0 .. kMxSpan: it and itself + 15 - kMxSpan in 0 .. 15, the bytes in two halves with a guard
  // bit above each
  constexpr uint32_t kMore = (15u - kMxSpan) * 0x10001u;
  const uint32_t d0 = ((st.ref & 0x00ff00ffu) | 0x01000100u) - (own & 0x00ff00ffu);
  const uint32_t d1 = (((st.ref >> 8) & 0x00ff00ffu) | 0x01000100u) - ((own >> 8) & 0x00ff00ffu);
  const bool fits = ((((d0 ^ 0x01000100u) | ((d0 + kMore) ^ 0x01000100u)) |
                      ((d1 ^ 0x01000100u) | ((d1 + kMore) ^ 0x01000100u))) & 0x01f001f0u) == 0u;
  bool fast = __all_sync(0xffffffffu, fits || !own_valid);
  if (!fast) {
    fast = mx_rebase(st, own, own_valid);
    const bool above = own_valid && (d0 & d1 & 0x01000100u) != 0x01000100u;  // some E_v > R, or NaN's 255
    if (!fast && __any_sync(0xffffffffu, above)) mx_follow(st, pa, pb, sv, key0, rows, 2 * (lane & 3), nh);
  }
  const uint32_t ref = st.ref;
  if (partial) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = kb + 2 * (lane & 3) + 8 * i;
      if (k >= rows) ev[i].x = ref;
      if (k + 1 >= rows) ev[i].y = ref;
    }
  }

  if (fast) {
    // f16 exponent fields E - R + 16 (1 .. 16 in each byte), moved to where they sit in a half's high byte
    const uint32_t base4 = (ref - 0x10101010u) << 2;
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const uint32_t p0 = movmatrix_trans(pack_f16x2(pa[2 * nb], pb[2 * nb]));
      const uint32_t p1 = movmatrix_trans(pack_f16x2(pa[2 * nb + 1], pb[2 * nb + 1]));
      const uint32_t pe = prmt(p0, p1, 0x5410u), po = prmt(p0, p1, 0x7632u);  // keys (2 t, 2 t + 8), (2 t + 1, 2 t + 9)
      const uint32_t e00 = ev[2 * nb].x * 4u - base4, e01 = ev[2 * nb].y * 4u - base4;
      const uint32_t e80 = ev[2 * nb + 1].x * 4u - base4, e81 = ev[2 * nb + 1].y * 4u - base4;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t r[4];
        ldmatrix_x4_trans(v_base + mx_at(row + 16 * nb, 2 * j + ch), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int b = 2 * j + i;
          // byte b of both words in the halves' high bytes; the low ones: a sign, 0
          constexpr uint32_t kSel[4] = {0x4808u, 0x5818u, 0x6828u, 0x7838u};
          const uint32_t q0 = hmul2(pe, prmt(e00, e80, kSel[b]));
          const uint32_t q1 = hmul2(po, prmt(e01, e81, kSel[b]));
          uint32_t ce[4], co[4];  // dims 0, 2 and 1, 3 of keys (2 t, 2 t + 8), then of (2 t + 1, 2 t + 9)
          e2m1x8_to_f16(even_nibbles(r[2 * i], r[2 * i + 1]), ce);
          e2m1x8_to_f16(odd_nibbles(r[2 * i], r[2 * i + 1]), co);
          mma_f16_16816(st.o[2 * b], ce[0], co[0], ce[2], co[2], q0, q1);
          mma_f16_16816(st.o[2 * b + 1], ce[1], co[1], ce[3], co[3], q0, q1);
        }
      }
    }
  } else {
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const uint32_t p0 = movmatrix_trans(pack_bf16x2(pa[2 * nb], pb[2 * nb]));
      const uint32_t p1 = movmatrix_trans(pack_bf16x2(pa[2 * nb + 1], pb[2 * nb + 1]));
      const uint32_t pe = prmt(p0, p1, 0x5410u), po = prmt(p0, p1, 0x7632u);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t r[4];
        ldmatrix_x4_trans(v_base + mx_at(row + 16 * nb, 2 * j + ch), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int b = 2 * j + i, sh = 8 * b;
          const uint32_t rb = (ref >> sh) & 255u;
          const uint2 e0 = ev[2 * nb], e8 = ev[2 * nb + 1];
          const uint32_t q0 =
              bmul2(pe, mx_bf16_scale((e0.x >> sh) & 255u, rb) | (mx_bf16_scale((e8.x >> sh) & 255u, rb) << 16));
          const uint32_t q1 =
              bmul2(po, mx_bf16_scale((e0.y >> sh) & 255u, rb) | (mx_bf16_scale((e8.y >> sh) & 255u, rb) << 16));
          uint32_t ce[4], co[4];
          e2m1x8_to_f16(even_nibbles(r[2 * i], r[2 * i + 1]), ce);
          e2m1x8_to_f16(odd_nibbles(r[2 * i], r[2 * i + 1]), co);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            ce[u] = f16x2_to_bf16x2(ce[u]);
            co[u] = f16x2_to_bf16x2(co[u]);
          }
          mma_bf16_16816(st.o[2 * b], ce[0], co[0], ce[2], co[2], q0, q1);
          mma_bf16_16816(st.o[2 * b + 1], ce[1], co[1], ce[3], co[3], q0, q1);
        }
      }
    }
  }
}

__device__ __forceinline__ void mx_consumer_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(kMxWarps * 32) : "memory");
}

// End of a work item: the warps' states merged, then the output (the
// unit's only split) or the split's partial.
__device__ __forceinline__ void mx_epilogue(const DecodeParams& p, const ItemCoord& c, const MxState& st, float* merge,
                                            bool single, int tid, int warp, int lane) {
  constexpr int D = kMxD;
  float* red_m = merge;
  float* red_l = red_m + kMxWarps * kDecHeadsPerCta;
  float* red_o = red_l + kMxWarps * kDecHeadsPerCta;
  float* ow = red_o + warp * kDecHeadsPerCta * D;
  mx_consumer_bar();  // the previous item's scratch has been read
  float l_a = st.l_a, l_b = st.l_b;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l_a += __shfl_xor_sync(0xffffffffu, l_a, off);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, off);
  }
  const int ha = 2 * (lane & 3);
  constexpr uint32_t kBias = (uint32_t)kMxBias;
  if (lane < 4) {
    const float f = __uint_as_float((127u - kBias) << 23);
    red_m[warp * 8 + ha] = st.m_a;
    red_m[warp * 8 + ha + 1] = st.m_b;
    red_l[warp * 8 + ha] = l_a * f;
    red_l[warp * 8 + ha + 1] = l_b * f;
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    // 2^(R - 127) / 2^(kMxBias + 1): large values are not to overflow before the division by l
    const float f = __uint_as_float((((st.ref >> (8 * b)) & 255u) - 1u - kBias) << 23);
    const int dim = 32 * b + 4 * (lane >> 2);
    const float* o0 = st.o[2 * b];
    const float* o1 = st.o[2 * b + 1];
    *reinterpret_cast<float4*>(ow + ha * D + dim) = make_float4(o0[0] * f, o0[2] * f, o1[0] * f, o1[2] * f);
    *reinterpret_cast<float4*>(ow + (ha + 1) * D + dim) = make_float4(o0[1] * f, o0[3] * f, o1[1] * f, o1[3] * f);
  }
  mx_consumer_bar();
  __nv_bfloat16* out_row = static_cast<__nv_bfloat16*>(p.out) + ((size_t)c.b * p.H + c.h0) * D;
  const size_t part = ((size_t)c.unit * p.nsplit + c.split) * p.G + (size_t)c.hsl * kDecHeadsPerCta;
  // four dims a thread
  for (int i = tid; i < c.nh * (D / 4); i += kMxWarps * 32) {
    const int h = i / (D / 4), dim = i % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kMxWarps; ++w) M = fmaxf(M, red_m[w * 8 + h]);
    const float ref = M == -INFINITY ? 0.f : M;  // every score of the item below float32's range, or NaN: 0, or NaN
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kMxWarps; ++w) {
      const float f = fast_exp2(red_m[w * 8 + h] - ref);
      const float4 v = *reinterpret_cast<const float4*>(red_o + (w * kDecHeadsPerCta + h) * D + dim);
      L = fmaf(red_l[w * 8 + h], f, L);
      O.x = fmaf(v.x, f, O.x);
      O.y = fmaf(v.y, f, O.y);
      O.z = fmaf(v.z, f, O.z);
      O.w = fmaf(v.w, f, O.w);
    }
    if (single) {
      if (L == 0.f) L = 1.f;  // no weight: zeros, as without keys
      *reinterpret_cast<uint2*>(out_row + h * D + dim) =
          make_uint2(pack_bf16x2(O.x / L, O.y / L), pack_bf16x2(O.z / L, O.w / L));
    } else {
      *reinterpret_cast<float4*>(p.ws_o + (part + h) * D + dim) = O;
      if (dim == 0) p.ws_ml[part + h] = make_float2(M, L);
    }
  }
}

__global__ void __launch_bounds__(kMxDecThreads, kMxCtasPerSm)
    decode_mxfp4_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                        const DecodeParams p, const MxParams mp) {
  using C = MxCfg;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + C::kMergeOff);
  StageInfo* info = reinterpret_cast<StageInfo*>(smem + C::kInfoOff);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + kMxStages;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023u) {  // the swizzle pattern needs aligned stages
    grid_dep_wait();
    if (threadIdx.x == 0) raise_error(GQA_DEVERR_TIMEOUT);
    return;
  }
  // before the grid dependency, as in decode_bf16_kernel: barriers, descriptors, an L2 warm-up (a hint) of the
  // first work item's codes, sized by a length that may be stale
  int spec_first = 0;
  if (warp == kMxWarps && lane == 0) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    prefetch_tensormap(&tm_k16);
    prefetch_tensormap(&tm_v16);
    if ((int)blockIdx.x < p.nitems) spec_first = __ldcg(p.seqlens + item_coord(p, blockIdx.x).b);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMxWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == kMxWarps && lane == 0 && (int)blockIdx.x < p.nitems)
    warm_first_item<kMxRowBytes>(p, item_coord(p, blockIdx.x), spec_first, kMxStages * kMxTileKeys);
  grid_dep_wait();
  grid_dep_launch();

  if (warp == kMxWarps) {
    if (lane != 0) return;
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
          uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)c.b * p.H + c.h0) * kMxD);
          for (int i = 0; i < c.nh * kMxD / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const int ntiles = (t_end - t_begin + kMxTileKeys - 1) / kMxTileKeys;
      for (int tt = 0; tt < ntiles; ++tt, ++it) {
        const int s = it % kMxStages;
        const int t0 = t_begin + tt * kMxTileKeys;
        const int rows = min(kMxTileKeys, t_end - t0);
        if (it >= kMxStages) ok = mbar_wait_bounded(&empty[s], ((it / kMxStages) - 1) & 1);
        if (!ok) break;
        info[s] = StageInfo{item, rows,
                            (tt == 0 ? kTileFirst : 0) | (tt == ntiles - 1 ? kTileLast : 0) |
                                (len <= p.chunk ? kUnitSingleSplit : 0),
                            -1};
        uint8_t* stage = smem + s * C::kStageBytes;
        const uint32_t sbytes = (uint32_t)((rows + 3) / 4 * 16);  // S_max is a multiple of 4: within the unit's scales
        const uint32_t q_bytes = tt == 0 ? (uint32_t)(c.nh * kMxD * 2) : 0u;
        const int row0 = c.unit * p.S_max + t0;
        if (rows == kMxTileKeys) {
          mbar_arrive_expect_tx(&full[s], 2u * C::kCodeBytes + 2u * sbytes + q_bytes);
          tma_load_2d(stage, &tm_k, 0, row0 / 2, &full[s], policy);
          tma_load_2d(stage + C::kCodeBytes, &tm_v, 0, row0 / 2, &full[s], policy);
        } else {
          const int nbox = (rows + kDecBoxRows - 1) / kDecBoxRows;
          mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * nbox * kDecBoxRows * kMxRowBytes) + 2u * sbytes + q_bytes);
          for (int bx = 0; bx < nbox; ++bx) {
            const int off = bx * kDecBoxRows * kMxRowBytes;
            tma_load_2d(stage + off, &tm_k16, 0, (row0 + bx * kDecBoxRows) / 2, &full[s], policy);
            tma_load_2d(stage + C::kCodeBytes + off, &tm_v16, 0, (row0 + bx * kDecBoxRows) / 2, &full[s], policy);
          }
        }
        bulk_load(stage + C::kScaleOff, mp.k_scales + (size_t)row0 * kMxScales, sbytes, &full[s]);
        bulk_load(stage + C::kScaleOff + kMxTileKeys * 4, mp.v_scales + (size_t)row0 * kMxScales, sbytes, &full[s]);
        if (q_bytes)
          bulk_load(stage + C::kQOff, static_cast<const __nv_bfloat16*>(p.q) + ((size_t)c.b * p.H + c.h0) * kMxD,
                    q_bytes, &full[s]);
      }
      if (!ok) break;
    }
    leave_queue(p.ws_queue, p.tag);
    if (ok) {  // a record without loads ends the consumers' loop
      const int s = it % kMxStages;
      if (it >= kMxStages) ok = mbar_wait_bounded(&empty[s], ((it / kMxStages) - 1) & 1);
      if (ok) {
        info[s] = StageInfo{-1, 0, 0, 0};
        mbar_arrive(&full[s]);
        ++it;
      }
    }
    // this CTA's own loads must land before the block may exit
    for (int j = max(0, it - kMxStages); j < it; ++j) mbar_wait_bounded(&full[j % kMxStages], (j / kMxStages) & 1);
    return;
  }

  const int tid = threadIdx.x;
  const int kb = warp * kMxWarpKeys;
  uint32_t qf[kMxD / 16][2];
  float f_a = 0.f, f_b = 0.f;
  MxState st;
  ItemCoord cur{};
  for (int it = 0;; ++it) {
    const int s = it % kMxStages;
    if (!mbar_wait_bounded(&full[s], (it / kMxStages) & 1)) break;
    const StageInfo si = info[s];
    if (si.item < 0) break;
    const uint8_t* stage = smem + s * C::kStageBytes;
    if (si.flags & kTileFirst) {
      cur = item_coord(p, si.item);
      const float up =
          load_q_frag_mx(qf, reinterpret_cast<const __nv_bfloat16*>(stage + C::kQOff), lane, cur.nh) * p.scale_log2;
      f_a = __shfl_sync(0xffffffffu, up, 8 * (lane & 3));
      f_b = __shfl_sync(0xffffffffu, up, 8 * (lane & 3) + 4);
      st.reset();
    }
    if (kb < si.rows) warp_tile_mx(st, qf, f_a, f_b, stage, kb, si.rows, lane, cur.nh);
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (si.flags & kTileLast) mx_epilogue(p, cur, st, merge, (si.flags & kUnitSingleSplit) != 0, tid, warp, lane);
  }
}

}  // namespace gqa
