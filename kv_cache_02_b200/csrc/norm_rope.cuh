// gqa_qk_norm_rope: the norm of each query and key head, the position
// rotation and the cache write, in one pass over the new tokens' rows.
//
//   y = x / sqrt(mean x^2 + eps) * w
//   (y_i, y_j) -> (y_i cos - y_j sin, y_j cos + y_i sin)
//
// A stream: every row is read once and written once (16-byte accesses), about
// 8 operations a value, so DRAM bounds a prompt and the launch a decode step.
// D / VEC lanes hold one row (16 lanes for d = 128 bf16); a lane keeps the
// cosines and sines of its dims for all rows of its token that it works on,
// since the heads of a token share them: read per row they would be twice the
// row's own bytes in L1 traffic. A rotation partner half a row away comes
// from its lane by one shuffle, so a row is complete in registers before it
// is written, and q_out may be q.
#pragma once

#include "common.cuh"

namespace gqa {

struct NormRopeParams {
  const void *q, *k, *v;
  void *q_out, *k_out;      // k_out may be null
  void *k_cache, *v_cache;  // or both null
  int32_t* row_pos;         // or null
  const void *q_weight, *k_weight;  // or null: no norm
  const float* rope;
  const int32_t *positions, *rows, *block_table;  // block_table: the paged form
  long long q_stride, k_stride, v_stride;         // elements between tokens
  int B, T, H, K, S_max, rotary_dim, max_pos, chunks;
  int num_blocks, block_size, max_blocks;
  float eps;
};

template <typename T>
struct Vec16 {
  static constexpr int N = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack16(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack16(const uint4& w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x);
  x[1] = __uint_as_float(w.y);
  x[2] = __uint_as_float(w.z);
  x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ uint4 pack16(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack16(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

constexpr int kNrThreads = 256;

// R: rows of a token that a lane group has in flight at once.
template <typename T, int D, bool kInterleaved, int R>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int VEC = Vec16<T>::N;
  constexpr int LPR = D / VEC;  // lanes per row
  constexpr int CPR = D / VEC;  // 16-byte chunks per row
  grid_dep_wait();
  grid_dep_launch();
  const int nrows = p.H + p.K + (p.v_cache ? p.K : 0);  // rows of a token
  const long long tokens = (long long)p.B * p.T;
  const long long group = (blockIdx.x * (long long)kNrThreads + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  const bool live = group < tokens * p.chunks;
  const long long n = live ? group / p.chunks : 0;
  const int chunk = (int)(live ? group % p.chunks : 0);
  const int b = (int)(n / p.T), t = (int)(n % p.T);
  // this chunk's rows of the token: chunk, chunk + chunks, ...

  int pos = p.positions ? p.positions[n] : 0;
  if (p.row_pos != nullptr || p.v_cache != nullptr) {
    const int row = p.rows[b] + t;
    const bool fits = p.rows[b] >= 0 && p.rows[b] <= p.S_max - p.T;
    if (live && !fits && chunk == 0 && t == 0 && l == 0) raise_error(GQA_DEVERR_APPEND_POS);
    if (live && fits && p.row_pos != nullptr && chunk == 0)
      for (int g = l; g < p.K; g += LPR) p.row_pos[((size_t)b * p.K + g) * p.S_max + row] = pos;
  }

  const int rd = p.rotary_dim;
  float cs[VEC], sn[VEC];
  int partner = l;
  const bool turns = l * VEC < rd;  // the lane's dims are rotated: all or none of them
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (rd > 0) {
    if (pos < 0 || pos >= p.max_pos) {
      if (live && chunk == 0 && l == 0) raise_error(GQA_DEVERR_ROPE_POS);
      pos = min(max(pos, 0), p.max_pos - 1);
    }
    const float* row = p.rope + (size_t)pos * rd;
    const int d0 = l * VEC;  // the lane's first dim
    if (d0 < rd) {
      if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {  // pair (2 j, 2 j + 1), j = d0 / 2 + i
          cs[2 * i] = cs[2 * i + 1] = __ldg(row + d0 / 2 + i);
          const float s = __ldg(row + rd / 2 + d0 / 2 + i);
          sn[2 * i] = -s;
          sn[2 * i + 1] = s;
        }
      } else {
        const bool upper = d0 >= rd / 2;  // a lane's dims lie in one half: rd / 2 is a multiple of VEC
        const int i0 = upper ? d0 - rd / 2 : d0;
        partner = upper ? l - rd / 2 / VEC : l + rd / 2 / VEC;
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
          const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + rd / 2 + i0 + i));
          cs[i] = c4.x, cs[i + 1] = c4.y, cs[i + 2] = c4.z, cs[i + 3] = c4.w;
          sn[i] = upper ? s4.x : -s4.x, sn[i + 1] = upper ? s4.y : -s4.y;
          sn[i + 2] = upper ? s4.z : -s4.z, sn[i + 3] = upper ? s4.w : -s4.w;
        }
      }
    }
  }

  // the token's cache row (chunks of 16 bytes), or -1
  long long crow = -1;
  long long crow_step = 0;  // chunks between KV heads
  if (p.v_cache != nullptr && p.rows[b] >= 0 && p.rows[b] <= p.S_max - p.T) {
    const int row = p.rows[b] + t;
    if (p.block_table == nullptr) {
      crow = ((long long)b * p.K * p.S_max + row) * CPR;
      crow_step = (long long)p.S_max * CPR;
    } else {
      const int blk = __ldg(p.block_table + (size_t)b * p.max_blocks + row / p.block_size);
      if ((unsigned)blk < (unsigned)p.num_blocks) {
        crow = ((long long)blk * p.K * p.block_size + row % p.block_size) * CPR;
        crow_step = (long long)p.block_size * CPR;
      } else if (live && chunk == 0 && l == 0) {
        raise_error(GQA_DEVERR_BLOCK);
      }
    }
  }

  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + n * p.q_stride);
  const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + n * p.k_stride);
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + (p.v ? n * p.v_stride : 0));
  uint4* q_out = static_cast<uint4*>(p.q_out) + n * p.H * CPR;
  uint4* k_out = p.k_out ? static_cast<uint4*>(p.k_out) + n * p.K * CPR : nullptr;

  // the loop count is the same for every lane of the warp: the shuffles are warp-wide
  const int rounds = (nrows + p.chunks * R - 1) / (p.chunks * R);
  for (int it = 0; it < rounds; ++it) {
    uint4 w[R];
    int row[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      row[r] = chunk + (it * R + r) * p.chunks;
      if (!live) row[r] = nrows;
      w[r] = make_uint4(0u, 0u, 0u, 0u);
      if (row[r] < p.H)
        w[r] = q[row[r] * CPR + l];
      else if (row[r] < p.H + p.K)
        w[r] = k[(row[r] - p.H) * CPR + l];
      else if (row[r] < nrows)
        w[r] = v[(row[r] - p.H - p.K) * CPR + l];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool is_q = row[r] < p.H, is_k = !is_q && row[r] < p.H + p.K;
      uint4 y = w[r];
      {
        float x[VEC];
        unpack16(w[r], x);
        const void* wt = is_q ? p.q_weight : p.k_weight;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, LPR);
        if (wt != nullptr) {
          const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
          float wv[VEC];
          unpack16(__ldg(static_cast<const uint4*>(wt) + l), wv);
#pragma unroll
          for (int i = 0; i < VEC; ++i) x[i] = x[i] * inv * wv[i];
        }
        float z[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float o = kInterleaved ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], partner, LPR);
          z[i] = turns ? x[i] * cs[i] + o * sn[i] : x[i];
        }
        if (is_q || is_k) y = pack16(z);
      }
      if (is_q) {
        q_out[row[r] * CPR + l] = y;
      } else if (is_k) {
        const int g = row[r] - p.H;
        if (k_out != nullptr) k_out[g * CPR + l] = y;
        if (crow >= 0) static_cast<uint4*>(p.k_cache)[crow + g * crow_step + l] = y;
      } else if (row[r] < nrows && crow >= 0) {
        static_cast<uint4*>(p.v_cache)[crow + (row[r] - p.H - p.K) * crow_step + l] = y;
      }
    }
  }
}

// gqa_rope_table: one thread per angle, in 64 bits.
__global__ void rope_table_kernel(float* __restrict__ rope, int max_pos, int half, double theta) {
  const long long total = (long long)max_pos * half;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int j = (int)(i % half);
    const long long pos = i / half;
    double s, c;
    sincos((double)pos * pow(theta, -(double)j / half), &s, &c);
    rope[pos * 2 * half + j] = (float)c;
    rope[pos * 2 * half + half + j] = (float)s;
  }
}

}  // namespace gqa
