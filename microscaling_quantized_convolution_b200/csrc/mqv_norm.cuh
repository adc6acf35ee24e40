// Layer norm over the channels of a [P][C][N] tensor, forward and backward.
//   mean = sum_c x / C, rstd = (sum_c (x - mean)^2 / C + eps)^(-1/2),
//   y = (x - mean)·rstd·gamma + beta;
//   with xh = (x - mean)·rstd and g = gamma·gy:
//   gx = rstd·(g - sum_c g / C - xh·sum_c (g·xh) / C),
//   ggamma[c] = sum_{p,n} gy·xh, gbeta[c] = sum_{p,n} gy.
// Memory-bound: each tensor is read once into registers and written once.
// The variance is summed around the mean (a second pass over the registers),
// so a large common offset costs no precision; all sums are fp32.
//   - Rows (N = 1): a block takes a row at a time, a thread K vectors of V
//     consecutive channels.
//   - Columns (N > 1): a block takes the C x TN tile of one position and TN
//     batch items; a thread K vectors of V batch items, R channels apart, so
//     a warp's loads are runs of whole tile rows.
// The backward blocks run over many rows or tiles and keep their channels'
// parameter gradients in registers; each block writes one partial row, and
// column_sum_kernel adds the rows in a fixed order.
#pragma once

#include "mqv_layer_common.cuh"

namespace mqv {

constexpr int kLnMaxThreads = 1024;
constexpr int kLnFewThreads = 256;   // blocks up to this size may use more registers: the T of the kernels

struct LnArgs {
  int64_t P, N;
  int C;
  float eps;
  const float *gamma, *beta;   // null: 1 and 0
  float *mean, *rstd;          // [P][N]; null in the forward pass: not kept
  TensorIn x, gy;
  TensorOut out;               // y, or gx
  float* part;                 // backward: [gridDim.x][2][C]; null: no parameter gradients
  // columns
  int tn, tiles;               // batch items per tile, tiles along the batch
  int lanes, rows;             // threads along a tile row, channels per step
};

// Sum over the block; every thread gets it.  buf: 33 floats.
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();               // buf free
  if (lane == 0) buf[w] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.f);
}

template <int V, int K>
__device__ __forceinline__ void load_row(const TensorIn& t, int64_t base, int C, float (&v)[K][V]) {
  if (t.bf16) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * V;
      if (c < C) load_bf16<V>(t.p, base + c, v[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * V;
      if (c < C) load_f32<V>(t.p, base + c, v[k]);
    }
  }
}

template <int V, int K, int T>
__global__ void __launch_bounds__(T) ln_fwd_row_kernel(const LnArgs a) {
  __shared__ float buf[33];
  const int C = a.C;
  const float inv = 1.f / C;
  for (int64_t p = blockIdx.x; p < a.P; p += gridDim.x) {
    float v[K][V];
    load_row<V, K>(a.x, p * C, C, v);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((threadIdx.x + k * blockDim.x) * V < C)
#pragma unroll
        for (int e = 0; e < V; ++e) s += v[k][e];
    const float mean = block_sum(s, buf) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if ((threadIdx.x + k * blockDim.x) * V < C)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          v[k][e] -= mean;
          s += v[k][e] * v[k][e];
        }
    const float rstd = 1.f / sqrtf(block_sum(s, buf) * inv + a.eps);
    if (threadIdx.x == 0 && a.mean) {
      a.mean[p] = mean;
      a.rstd[p] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * V;
      if (c < C) {
        float g[V], b[V];
        if (a.gamma) load_f32<V>(a.gamma, c, g);
        if (a.beta) load_f32<V>(a.beta, c, b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float y = v[k][e] * rstd;
          if (a.gamma) y *= g[e];
          if (a.beta) y += b[e];
          v[k][e] = y;
        }
        store_vec<V>(a.out, p * C + c, v[k]);
      }
    }
  }
}

template <int V, int K, int T>
__global__ void __launch_bounds__(T) ln_bwd_row_kernel(const LnArgs a) {
  __shared__ float buf[2][33];
  const int C = a.C;
  const float inv = 1.f / C;
  float ag[K][V], ab[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) ag[k][e] = ab[k][e] = 0.f;
  for (int64_t p = blockIdx.x; p < a.P; p += gridDim.x) {
    float x[K][V], g[K][V];
    load_row<V, K>(a.x, p * C, C, x);
    load_row<V, K>(a.gy, p * C, C, g);
    const float mean = a.mean[p], rstd = a.rstd[p];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * V;
      if (c < C) {
        float w[V];
        if (a.gamma) load_f32<V>(a.gamma, c, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[k][e] = (x[k][e] - mean) * rstd;
          ag[k][e] += g[k][e] * x[k][e];
          ab[k][e] += g[k][e];
          if (a.gamma) g[k][e] *= w[e];
          s1 += g[k][e];
          s2 += g[k][e] * x[k][e];
        }
      }
    }
    s1 = block_sum(s1, buf[0]) * inv;
    s2 = block_sum(s2, buf[1]) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * V;
      if (c < C) {
#pragma unroll
        for (int e = 0; e < V; ++e) g[k][e] = rstd * (g[k][e] - s1 - x[k][e] * s2);
        store_vec<V>(a.out, p * C + c, g[k]);
      }
    }
  }
  if (a.part) {
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (threadIdx.x + k * blockDim.x) * V;
      if (c < C)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          part[c + e] = ag[k][e];
          part[C + c + e] = ab[k][e];
        }
    }
  }
}

// Sums the V values of the threads that share a tile column (same thread
// index modulo `lanes`) over the block's channel rows; every active thread
// gets its column's sums.  buf: blockDim.x·V floats.
template <int V>
__device__ __forceinline__ void tile_sum(float (&v)[V], int lanes, int rows, float* buf) {
  const int t = threadIdx.x, r = t / lanes;
  const bool act = r < rows;
  __syncthreads();               // buf free
  if (act)
#pragma unroll
    for (int e = 0; e < V; ++e) buf[e * blockDim.x + t] = v[e];
  for (int n = rows; n > 1;) {
    const int half = (n + 1) / 2;
    __syncthreads();
    if (r < n - half)
#pragma unroll
      for (int e = 0; e < V; ++e) buf[e * blockDim.x + t] += buf[e * blockDim.x + t + half * lanes];
    n = half;
  }
  __syncthreads();
  if (act)
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = buf[e * blockDim.x + t % lanes];
}

template <int V, int K>
__device__ __forceinline__ void load_tile(const TensorIn& t, int64_t base, int64_t N, int r, int rows, int C, bool act,
                                          float (&v)[K][V]) {
  if (t.bf16) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (act && r + k * rows < C) load_bf16<V>(t.p, base + (r + k * rows) * N, v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (act && r + k * rows < C) load_f32<V>(t.p, base + (r + k * rows) * N, v[k]);
  }
}

template <int V, int K, int T>
__global__ void __launch_bounds__(T) ln_fwd_tile_kernel(const LnArgs a) {
  extern __shared__ float buf[];
  const int C = a.C, r = threadIdx.x / a.lanes, l = threadIdx.x % a.lanes;
  const float inv = 1.f / C;
  const int64_t total = a.P * a.tiles;
  for (int64_t s = blockIdx.x; s < total; s += gridDim.x) {
    const int64_t p = s / a.tiles, n = (s % a.tiles) * a.tn + l * V;
    const bool act = r < a.rows && n < a.N;
    const int64_t base = p * C * a.N + n;
    float v[K][V], m[V], q[V];
    load_tile<V, K>(a.x, base, a.N, r, a.rows, C, act, v);
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] = q[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (act && r + k * a.rows < C)
#pragma unroll
        for (int e = 0; e < V; ++e) m[e] += v[k][e];
    tile_sum<V>(m, a.lanes, a.rows, buf);
#pragma unroll
    for (int e = 0; e < V; ++e) m[e] *= inv;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (act && r + k * a.rows < C)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          v[k][e] -= m[e];
          q[e] += v[k][e] * v[k][e];
        }
    tile_sum<V>(q, a.lanes, a.rows, buf);
#pragma unroll
    for (int e = 0; e < V; ++e) q[e] = 1.f / sqrtf(q[e] * inv + a.eps);
    if (act && r == 0 && a.mean)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        a.mean[p * a.N + n + e] = m[e];
        a.rstd[p * a.N + n + e] = q[e];
      }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = r + k * a.rows;
      if (act && c < C) {
        const float g = a.gamma ? __ldg(a.gamma + c) : 1.f, b = a.beta ? __ldg(a.beta + c) : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = v[k][e] * q[e] * g + b;
        store_vec<V>(a.out, base + c * a.N, v[k]);
      }
    }
  }
}

template <int V, int K, int T>
__global__ void __launch_bounds__(T) ln_bwd_tile_kernel(const LnArgs a) {
  extern __shared__ float buf[];
  const int C = a.C, r = threadIdx.x / a.lanes, l = threadIdx.x % a.lanes;
  const float inv = 1.f / C;
  const int64_t total = a.P * a.tiles;
  float ag[K], ab[K];
#pragma unroll
  for (int k = 0; k < K; ++k) ag[k] = ab[k] = 0.f;
  for (int64_t s = blockIdx.x; s < total; s += gridDim.x) {
    const int64_t p = s / a.tiles, n = (s % a.tiles) * a.tn + l * V;
    const bool act = r < a.rows && n < a.N;
    const int64_t base = p * C * a.N + n;
    float x[K][V], g[K][V], m[V], q[V], s1[V], s2[V];
    load_tile<V, K>(a.x, base, a.N, r, a.rows, C, act, x);
    load_tile<V, K>(a.gy, base, a.N, r, a.rows, C, act, g);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      m[e] = act ? a.mean[p * a.N + n + e] : 0.f;
      q[e] = act ? a.rstd[p * a.N + n + e] : 0.f;
      s1[e] = s2[e] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = r + k * a.rows;
      if (act && c < C) {
        const float w = a.gamma ? __ldg(a.gamma + c) : 1.f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[k][e] = (x[k][e] - m[e]) * q[e];
          ag[k] += g[k][e] * x[k][e];
          ab[k] += g[k][e];
          g[k][e] *= w;
          s1[e] += g[k][e];
          s2[e] += g[k][e] * x[k][e];
        }
      }
    }
    tile_sum<V>(s1, a.lanes, a.rows, buf);
    tile_sum<V>(s2, a.lanes, a.rows, buf);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = r + k * a.rows;
      if (act && c < C) {
#pragma unroll
        for (int e = 0; e < V; ++e) g[k][e] = q[e] * (g[k][e] - s1[e] * inv - x[k][e] * (s2[e] * inv));
        store_vec<V>(a.out, base + c * a.N, g[k]);
      }
    }
  }
  if (a.part) {
    // a channel's sums over the lanes of its row, added in lane order
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      __syncthreads();
      buf[threadIdx.x] = ag[k];
      buf[blockDim.x + threadIdx.x] = ab[k];
      __syncthreads();
      const int c = r + k * a.rows;
      if (l < 2 && r < a.rows && c < C) {
        for (int h = l; h < 2; h += a.lanes) {
          float t = 0.f;
          for (int i = 0; i < a.lanes; ++i) t += buf[h * blockDim.x + r * a.lanes + i];
          part[h * C + c] = t;
        }
      }
    }
  }
}

}  // namespace mqv
