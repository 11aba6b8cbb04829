// Rows of the 4-bit cache: quantizing append and read-back.
//
// A block of 32 values x is held as codes e2m1(x / 2^(E - 127)) and the
// exponent E = floor(log2 max|x|) - 2 + 127. Both are exact integer work on
// the values' bits but for the one rounding of the code, which the hardware's
// conversion makes (nearest, ties to even, saturating).
//
// Streams: 16 lanes hold one row of 128 (8 values, one 16-byte access each),
// so a block is 4 lanes and its maximum two shuffles.
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

// The value of exponent E: 2^(E - 127), NaN for 255
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return e == 0 ? __uint_as_float(0x00400000u) : e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(e << 23);
}

// Row index r of the call (K rows of all tokens, then V rows) -> tensor, token, head.
__global__ void __launch_bounds__(kMxThreads)
    kv_append_mxfp4_kernel(uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                           const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                           const int32_t* __restrict__ pos, int B, int T, int K, int S_max) {
  grid_dep_wait();
  grid_dep_launch();
  const long long nrows = (long long)B * T * K;
  const int l = threadIdx.x & 15;
  const long long per_round = (long long)gridDim.x * (kMxThreads / 16);
  const long long rounds = (2 * nrows + per_round - 1) / per_round;
  for (long long it = 0; it < rounds; ++it) {
    const long long r = it * per_round + blockIdx.x * (long long)(kMxThreads / 16) + (threadIdx.x >> 4);
    const bool live = r < 2 * nrows;
    const bool is_v = r >= nrows;
    const long long row = live ? (is_v ? r - nrows : r) : 0;  // (b * T + t) * K + g
    const int g = (int)(row % K);
    const long long n = row / K;
    const int t = (int)(n % T), b = (int)(n / T);
    const int p0 = __ldg(pos + b);
    const uint4 w = live ? __ldg((is_v ? v_new : k_new) + row * 16 + l) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float x[8];
    uint32_t top = 0;  // the block's largest magnitude, as bits: a NaN's are above infinity's
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      top = max(top, max((u[i] << 16) & 0x7fffffffu, u[i] & 0x7fff0000u));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool bad = top >= 0x7f800000u;
    const uint32_t e = bad ? 255u : (uint32_t)max((int)(top >> 23) - 2, 0);
    const float inv = bad ? 0.f : __uint_as_float((254u - e) << 23);  // 2^(127 - E), exact
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bad ? 0.f : x[i] * inv;
    const uint32_t codes = e2m1x8(x);
    // the row's four scales in lane 0 of the 16
    uint32_t sc = e;
    sc |= __shfl_down_sync(0xffffffffu, sc, 4, 16) << 8;   // lanes 0, 8: two scales
    sc |= __shfl_down_sync(0xffffffffu, sc, 8, 16) << 16;  // lane 0: four
    if (!live) continue;
    if (p0 < 0 || p0 > S_max - T) {
      if (l == 0 && !is_v && g == 0 && t == 0) raise_error(GQA_DEVERR_APPEND_POS);
      continue;
    }
    const long long dst = ((long long)b * K + g) * S_max + p0 + t;
    reinterpret_cast<uint32_t*>((is_v ? v_codes : k_codes) + dst * kMxRowBytes)[l] = codes;
    if (l == 0) reinterpret_cast<uint32_t*>(is_v ? v_scales : k_scales)[dst] = sc;
  }
}

// 8 e2m1 codes -> bf16 values times the scale, exact
__device__ __forceinline__ uint4 mx_values8(uint32_t codes, float scale) {
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t c = codes >> (8 * i + 4 * j);
      // the code's exponent and mantissa bits at the top of an fp16 one: value * 2^-14
      const uint32_t h = ((c & 7u) << 9) | ((c & 8u) << 12);
      v[j] = __half2float(__ushort_as_half((unsigned short)h)) * 16384.f * scale;
    }
    out[i] = pack_bf16x2(v[0], v[1]);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

__global__ void __launch_bounds__(kMxThreads)
    kv_read_mxfp4_kernel(uint4* __restrict__ k_out, uint4* __restrict__ v_out, const uint8_t* __restrict__ k_codes,
                         const uint8_t* __restrict__ k_scales, const uint8_t* __restrict__ v_codes,
                         const uint8_t* __restrict__ v_scales, const int32_t* __restrict__ pos, int B, int T, int K,
                         int S_max) {
  grid_dep_wait();
  grid_dep_launch();
  const long long nrows = (long long)B * T * K;
  const int l = threadIdx.x & 15;
  const long long per_round = (long long)gridDim.x * (kMxThreads / 16);
  for (long long r = blockIdx.x * (long long)(kMxThreads / 16) + (threadIdx.x >> 4); r < 2 * nrows; r += per_round) {
    const bool is_v = r >= nrows;
    const long long row = is_v ? r - nrows : r;
    const int g = (int)(row % K);
    const long long n = row / K;
    const int t = (int)(n % T), b = (int)(n / T);
    const int p0 = __ldg(pos + b);
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (p0 < 0 || p0 > S_max - T) {
      if (l == 0 && !is_v && g == 0 && t == 0) raise_error(GQA_DEVERR_APPEND_POS);
    } else {
      const long long src = ((long long)b * K + g) * S_max + p0 + t;
      const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>((is_v ? v_codes : k_codes) + src * kMxRowBytes) + l);
      const uint32_t sc = __ldg(reinterpret_cast<const uint32_t*>(is_v ? v_scales : k_scales) + src);
      val = mx_values8(codes, e8m0_value((sc >> (8 * (l >> 2))) & 255u));
    }
    (is_v ? v_out : k_out)[row * 16 + l] = val;
  }
}

}  // namespace gqa
