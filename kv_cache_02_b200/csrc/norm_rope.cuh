// gqa_qk_norm_rope: the norm of each query and key head, the position
// rotation and the cache write, in one pass over the new tokens' rows.
//
//   y = x / sqrt(mean x^2 + eps) * w
//   (y_i, y_j) -> (y_i cos - y_j sin, y_j cos + y_i sin)
//
// A stream: every row is read once and written once, about 8 operations a
// value, so DRAM bounds a prompt and the launch a decode step. D / 8 lanes
// hold one row, 8 values each as two chunks of 4 that are each other's
// rotation partners (i and i + rotary_dim / 2), so that the rotation needs no
// exchange between lanes and a lane's 4 cosines and sines serve 8 values. A
// group of lanes takes up to R rows of one token, which share that table row.
// The rows are asked for first: the table's address has to wait for the
// position. A row is complete in registers before it is written, so q_out may
// be q.
//
// Measured: 4 x 4096 tokens of 32 + 8 heads, d 128, bfloat16, no cache: 73 us,
// 4.70 TB/s, 0.72 of a copy; issue slots 70 % used at 7 warps a
// scheduler. R = 2 takes 125 us, 8 77 us, 5 81 us; persistent blocks that load
// the next token's rows ahead need 96 to 116 registers and take 80 to 115 us.
// With the cache write 93 us (0.68), into pages of 16 102 us; float32 108, 130
// and 142 us (0.96, 0.95, 0.88). A decode step of 8 tokens into a paged cache: 2.6
// us in a graph.
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

// Four values in memory
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
  static __device__ __forceinline__ void unpack(const Raw& w, float* x) {
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw pack(const float* x) {
    return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  }
};
template <>
struct Quad<float> {
  using Raw = float4;
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void unpack(const Raw& w, float* x) {
    x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
  }
  static __device__ __forceinline__ Raw pack(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};

constexpr int kNrThreads = 256;

template <typename T, int D, bool kInterleaved, int R>
__global__ void __launch_bounds__(kNrThreads) qk_norm_rope_kernel(const NormRopeParams p) {
  using Q = Quad<T>;
  using Raw = typename Q::Raw;
  constexpr int LPR = D / 8;  // lanes per row
  grid_dep_wait();
  grid_dep_launch();
  const int nrows = p.H + p.K + (p.v_cache ? p.K : 0);  // rows of a token
  const unsigned group = (blockIdx.x * (unsigned)kNrThreads + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  const bool live = group < (unsigned)(p.B * p.T) * (unsigned)p.chunks;
  const unsigned n = live ? group / (unsigned)p.chunks : 0u;
  const int chunk = live ? (int)(group - n * (unsigned)p.chunks) : nrows;  // rows R chunk, R chunk + 1, ...

  // the lane's two chunks of a row, and whether they are rotated (all 8 values or none)
  const int rd = p.rotary_dim;
  const bool turns = 8 * l < rd;
  int lo, hi;
  if (kInterleaved) {
    lo = 8 * l;
    hi = lo + 4;
  } else if (turns) {
    lo = 4 * l;
    hi = lo + rd / 2;
  } else {
    lo = rd + 4 * (l - rd / 8);
    hi = lo + (D - rd) / 2;
  }

  const T* q = static_cast<const T*>(p.q) + n * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + n * p.k_stride - (long long)p.H * D;
  const T* v = p.v_cache ? static_cast<const T*>(p.v) + n * p.v_stride - (long long)(p.H + p.K) * D : nullptr;
  Raw w[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = R * chunk + r;
    w[r][0] = w[r][1] = Q::zero();
    if (row < nrows) {
      const T* x = (row < p.H ? q : row < p.H + p.K ? k : v) + row * D;
      w[r][0] = *reinterpret_cast<const Raw*>(x + lo);
      w[r][1] = *reinterpret_cast<const Raw*>(x + hi);
    }
  }

  int pos = p.positions ? p.positions[n] : 0;
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  const int given = pos;
  if (rd > 0) {
    if (pos < 0 || pos >= p.max_pos) {
      if (chunk == 0 && l == 0) raise_error(GQA_DEVERR_ROPE_POS);
      pos = min(max(pos, 0), p.max_pos - 1);
    }
    if (turns) {
      const float* row = p.rope + (size_t)pos * rd + 4 * l;
      const float4 c4 = *reinterpret_cast<const float4*>(row);
      const float4 s4 = *reinterpret_cast<const float4*>(row + rd / 2);
      cs[0] = c4.x, cs[1] = c4.y, cs[2] = c4.z, cs[3] = c4.w;
      sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
    }
  }

  // the token's row in the cache (elements, head 0), or -1
  long long crow = -1, crow_step = 0;
  if (p.row_pos != nullptr || p.v_cache != nullptr) {
    const int b = (int)(n / (unsigned)p.T), t = (int)(n - (unsigned)b * (unsigned)p.T);
    const int first = p.rows[b];
    const bool fits = first >= 0 && first <= p.S_max - p.T;
    const int row = first + t;
    if (!fits) {
      if (chunk == 0 && t == 0 && l == 0) raise_error(GQA_DEVERR_APPEND_POS);
    } else {
      if (p.row_pos != nullptr && chunk == 0)
        for (int g = l; g < p.K; g += LPR) p.row_pos[((size_t)b * p.K + g) * p.S_max + row] = given;
      if (p.v_cache != nullptr) {
        if (p.block_table == nullptr) {
          crow = ((long long)b * p.K * p.S_max + row) * D;
          crow_step = (long long)p.S_max * D;
        } else {
          const int at = row / p.block_size;
          const int blk = __ldcg(p.block_table + (size_t)b * p.max_blocks + at);
          if ((unsigned)blk < (unsigned)p.num_blocks) {
            crow = ((long long)blk * p.K * p.block_size + (row - at * p.block_size)) * D;
            crow_step = (long long)p.block_size * D;
          } else if (chunk == 0 && l == 0) {
            raise_error(GQA_DEVERR_BLOCK);
          }
        }
      }
    }
  }

  auto put = [&](T* dst, const Raw (&y)[2]) {
    *reinterpret_cast<Raw*>(dst + lo) = y[0];
    *reinterpret_cast<Raw*>(dst + hi) = y[1];
  };
  const T* wt = nullptr;
  float wv[8];
  T* q_out = static_cast<T*>(p.q_out) + (long long)n * p.H * D;
  T* k_out = p.k_out ? static_cast<T*>(p.k_out) + (long long)n * p.K * D : nullptr;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = R * chunk + r;
    const bool is_q = row < p.H, is_k = !is_q && row < p.H + p.K;
    float x[8];
    Q::unpack(w[r][0], x);
    Q::unpack(w[r][1], x + 4);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, LPR);
    if (r == 0 || row == p.H) {
      wt = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
      if (wt != nullptr) {
        Q::unpack(*reinterpret_cast<const Raw*>(wt + lo), wv);
        Q::unpack(*reinterpret_cast<const Raw*>(wt + hi), wv + 4);
      }
    }
    if (wt != nullptr) {
      // as exact, here, as 1 / sqrtf, which takes 5 % more of a prompt's time in float32 (114 us against 108)
      const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wv[i];
    }
    if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : i + 4;
        const float a = x[ia], b = x[ib];
        x[ia] = a * cs[i] - b * sn[i];
        x[ib] = b * cs[i] + a * sn[i];
      }
    }
    const Raw y[2] = {Q::pack(x), Q::pack(x + 4)};
    if (is_q) {
      put(q_out + row * D, y);
    } else if (is_k) {
      const int g = row - p.H;
      if (k_out != nullptr) put(k_out + g * D, y);
      if (crow >= 0) put(static_cast<T*>(p.k_cache) + crow + g * crow_step, y);
    } else if (row < nrows && crow >= 0) {
      put(static_cast<T*>(p.v_cache) + crow + (row - p.H - p.K) * crow_step, w[r]);
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
