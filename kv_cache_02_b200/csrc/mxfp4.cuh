// Rows of the 4-bit cache: quantizing append and read-back.
//
// A block of 32 values x is held as codes e2m1(x / 2^(E - 127)) and the
// exponent E = floor(log2 max|x|) - 2 + 127. Both are exact integer work on
// the values' bits but for the one rounding of the code, which the hardware's
// conversion makes (nearest, ties to even, saturating).
//
// Streams: 8 lanes hold one row of 128, the 8 values of 16-byte chunk l and
// those of chunk l + 8 in lane l, so that every access is contiguous over the
// lanes and a block is four lanes; a lane group has kMxUnroll rows in flight.
// The grid's y dimension is sequence and tensor: one division by K is all the
// index arithmetic of a row. 4 x 4096 tokens, 8 KV heads: append 15 us, read 15
// us (26 us of bytes at a copy's rate for both).
#pragma once

#include "common.cuh"

namespace gqa {

constexpr int kMxD = 128;               // dims of a row
constexpr int kMxRowBytes = kMxD / 2;   // codes of a row
constexpr int kMxScales = kMxD / 32;    // scales of a row
constexpr int kMxThreads = 256;

// 8 floats -> 8 e2m1 codes, value i in bits 4 i .. 4 i + 3
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Maxima of the two unsigned halves
__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("max.u16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// 8 codes of a word -> 4 f16x2: r[i] = (code 2 i, code 2 i + 1)
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// f16x2 -> bf16x2; the e2m1 values are exact in both
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack_bf16x2(f.x, f.y);
}

// The value of exponent E, 2^(E - 127), NaN for 255, in both halves as bfloat16
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t e) {
  return (e == 0 ? 0x0040u : e == 255 ? 0x7fc0u : e << 7) * 0x10001u;
}

constexpr int kMxLanes = 8;    // lanes of a row
constexpr int kMxUnroll = 4;   // rows of a lane group
constexpr int kMxBlockRows = kMxThreads / kMxLanes * kMxUnroll;

// blockIdx.y: 2 b for K, 2 b + 1 for V; rows t * K + g of the sequence
__global__ void __launch_bounds__(kMxThreads)
    kv_append_mxfp4_kernel(uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                           const uint8_t* __restrict__ k_new, const uint8_t* __restrict__ v_new,
                           const int32_t* __restrict__ pos, int B, int T, int K, int S_max) {
  grid_dep_wait();
  grid_dep_launch();
  const unsigned nrows = (unsigned)T * (unsigned)K;
  const int l = threadIdx.x % kMxLanes;
  const unsigned r0 = blockIdx.x * (unsigned)kMxBlockRows + threadIdx.x / kMxLanes;
  for (int y = blockIdx.y; y < 2 * B; y += gridDim.y) {
    const bool is_v = y & 1;
    const int b = y >> 1;
    const int p0 = __ldcg(pos + b);
    const uint4* src = reinterpret_cast<const uint4*>((is_v ? v_new : k_new) + (size_t)b * nrows * (2 * kMxD)) + l;
    uint4 w[kMxUnroll][2];
#pragma unroll
    for (int i = 0; i < kMxUnroll; ++i) {
      const unsigned r = r0 + i * (kMxThreads / kMxLanes);
      w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (r < nrows) {
        w[i][0] = __ldcg(src + (size_t)r * 16);
        w[i][1] = __ldcg(src + (size_t)r * 16 + 8);
      }
    }
    const bool fits = p0 >= 0 && p0 <= S_max - T;
    if (!fits && !is_v && blockIdx.x == 0 && threadIdx.x == 0) raise_error(GQA_DEVERR_APPEND_POS);
#pragma unroll
    for (int i = 0; i < kMxUnroll; ++i) {
      const unsigned r = r0 + i * (kMxThreads / kMxLanes);
      uint32_t codes[2], e[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t u[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
        // the block's largest magnitude, as bits: a NaN's are above infinity's
        uint32_t top = umax2(umax2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu), umax2(u[2] & 0x7fff7fffu, u[3] & 0x7fff7fffu));
        top = umax2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = umax2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top & 0xffffu, top >> 16);
        const bool bad = top >= 0x7f80u;
        e[h] = bad ? 255u : (uint32_t)max((int)(top >> 7) - 2, 0);
        // times 2^(127 - E), in bfloat16: exact, but for values far below a quarter of the scale
        const uint32_t inv = bad ? 0u : ((254u - e[h]) << 7) * 0x10001u;
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v = bmul2(u[j], inv);
          x[2 * j] = __uint_as_float(v << 16);
          x[2 * j + 1] = __uint_as_float(v & 0xffff0000u);
        }
        codes[h] = bad ? 0u : e2m1x8(x);
      }
      // the row's four scales in lane 0: blocks 0, 2 are its own, 1, 3 those of lane 4
      uint32_t sc = e[0] | (e[1] << 16);
      sc |= __shfl_down_sync(0xffffffffu, sc, 4, kMxLanes) << 8;
      if (r < nrows && fits) {
        const unsigned t = r / (unsigned)K, g = r - t * (unsigned)K;
        const size_t dst = ((size_t)b * K + g) * S_max + p0 + t;
        uint32_t* row = reinterpret_cast<uint32_t*>((is_v ? v_codes : k_codes) + dst * kMxRowBytes);
        row[l] = codes[0];
        row[l + 8] = codes[1];
        if (l == 0) reinterpret_cast<uint32_t*>(is_v ? v_scales : k_scales)[dst] = sc;
      }
    }
  }
}

// 8 e2m1 codes times the scale -> bf16 values (one rounding, of results past bfloat16's ends alone)
__device__ __forceinline__ uint4 mx_values8(uint32_t codes, uint32_t scale) {
  uint32_t h[4];
  e2m1x8_to_f16(codes, h);
  return make_uint4(bmul2(f16x2_to_bf16x2(h[0]), scale), bmul2(f16x2_to_bf16x2(h[1]), scale),
                    bmul2(f16x2_to_bf16x2(h[2]), scale), bmul2(f16x2_to_bf16x2(h[3]), scale));
}

__global__ void __launch_bounds__(kMxThreads)
    kv_read_mxfp4_kernel(uint8_t* __restrict__ k_out, uint8_t* __restrict__ v_out, const uint8_t* __restrict__ k_codes,
                         const uint8_t* __restrict__ k_scales, const uint8_t* __restrict__ v_codes,
                         const uint8_t* __restrict__ v_scales, const int32_t* __restrict__ pos, int B, int T, int K,
                         int S_max) {
  grid_dep_wait();
  grid_dep_launch();
  const unsigned nrows = (unsigned)T * (unsigned)K;
  const int l = threadIdx.x % kMxLanes;
  const unsigned r0 = blockIdx.x * (unsigned)kMxBlockRows + threadIdx.x / kMxLanes;
  for (int y = blockIdx.y; y < 2 * B; y += gridDim.y) {
    const bool is_v = y & 1;
    const int b = y >> 1;
    const int p0 = __ldcg(pos + b);
    const bool fits = p0 >= 0 && p0 <= S_max - T;
    if (!fits && !is_v && blockIdx.x == 0 && threadIdx.x == 0) raise_error(GQA_DEVERR_APPEND_POS);
    uint4* out = reinterpret_cast<uint4*>((is_v ? v_out : k_out) + (size_t)b * nrows * (2 * kMxD)) + l;
    uint32_t codes[kMxUnroll][2], sc[kMxUnroll];
#pragma unroll
    for (int i = 0; i < kMxUnroll; ++i) {
      const unsigned r = r0 + i * (kMxThreads / kMxLanes);
      codes[i][0] = codes[i][1] = 0u;
      sc[i] = 0x7f7f7f7fu;
      if (r < nrows && fits) {
        const unsigned t = r / (unsigned)K, g = r - t * (unsigned)K;
        const size_t at = ((size_t)b * K + g) * S_max + p0 + t;
        const uint32_t* row = reinterpret_cast<const uint32_t*>((is_v ? v_codes : k_codes) + at * kMxRowBytes);
        codes[i][0] = __ldcg(row + l);
        codes[i][1] = __ldcg(row + l + 8);
        sc[i] = __ldcg(reinterpret_cast<const uint32_t*>(is_v ? v_scales : k_scales) + at);
      }
    }
#pragma unroll
    for (int i = 0; i < kMxUnroll; ++i) {
      const unsigned r = r0 + i * (kMxThreads / kMxLanes);
      if (r >= nrows) continue;
      const uint32_t mine = sc[i] >> (8 * (l >> 2));  // blocks l / 4 and l / 4 + 2
      out[(size_t)r * 16] = mx_values8(codes[i][0], e8m0_bf16x2(mine & 255u));
      out[(size_t)r * 16 + 8] = mx_values8(codes[i][1], e8m0_bf16x2((mine >> 16) & 255u));
    }
  }
}

}  // namespace gqa
