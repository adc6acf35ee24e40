// The matrix product over the channels of a [P][C][N] tensor, with bias,
// activation and residual in its epilogue, and its gradients:
//   z[co][j] = sum_ci w[co][ci]·x[ci][j] + bias[co],  y = act(z) + residual,
//   gz = gy·act'(z), gbias[co] = sum_j gz[co][j],
//   gx[ci][j] = sum_co w[co][ci]·gz[co][j],  gw[co][ci] = sum_j gz[co][j]·x[ci][j],
// where j runs over the columns (p, n) of the tensors.  Operands are
// bfloat16, sums fp32.
#pragma once

#include "mqv_layer_common.cuh"

namespace mqv {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;       // a NaN stays one
    case kActGelu: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case kActSilu: return z / (1.f + expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActGelu:
      return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * (0.3989422804014327f * expf(-0.5f * z * z));
    case kActSilu: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    default: return 1.f;
  }
}

// ------------------------------------------------ matrix product, one tile

// Element offset of index i of one dimension: whole groups of `div` apart by
// `outer`, items of a group apart by `inner`.
struct Dim {
  int64_t div, outer, inner;
  __host__ __device__ int64_t at(int64_t i) const { return (i / div) * outer + (i % div) * inner; }
};

struct GemmArgs {
  const uint16_t *a, *b;       // bf16
  Dim a_row, a_k, b_col, b_k;
  int64_t M, N, K;
  TensorOut d, z;              // z.p null: not kept
  const void* residual;        // of d's type; null: none
  Dim d_row, d_col;
  const float* bias;           // null: none
  int bias_on_row, act;
};

// D[m][n] = epilogue(sum_k A[m][k]·B[k][n]), 64 x 64 outputs a block, 4 x 4 a
// thread, K in steps of 16 through shared memory.
__global__ void __launch_bounds__(256) gemm_simple_kernel(const GemmArgs g) {
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tiles_n = (g.N + 63) / 64;
  const int64_t m0 = (blockIdx.x / tiles_n) * 64, n0 = (blockIdx.x % tiles_n) * 64;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < g.K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i & 63, k = i >> 6;
      const bool kin = k0 + k < g.K;
      sa[k][r] = kin && m0 + r < g.M
                     ? __uint_as_float(static_cast<uint32_t>(g.a[g.a_row.at(m0 + r) + g.a_k.at(k0 + k)]) << 16) : 0.f;
      sb[k][r] = kin && n0 + r < g.N
                     ? __uint_as_float(static_cast<uint32_t>(g.b[g.b_col.at(n0 + r) + g.b_k.at(k0 + k)]) << 16) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= g.M || n >= g.N) continue;
      const int64_t o = g.d_row.at(m) + g.d_col.at(n);
      float v = acc[i][j];
      if (g.bias) v += g.bias[g.bias_on_row ? m : n];
      if (g.z.p) store_vec<1>(g.z, o, {v});
      v = act_value(v, g.act);
      if (g.residual) {
        float r[1];
        g.d.bf16 ? load_bf16<1>(g.residual, o, r) : load_f32<1>(g.residual, o, r);
        v += r[0];
      }
      store_vec<1>(g.d, o, {v});
    }
}

// --------------------------------------- gradient of activation and bias

struct ActGradArgs {
  TensorIn gy;
  const void* z;               // bf16; null: no activation
  TensorOut gz;                // null: not written
  float* part;                 // [gridDim.y][C]; null: no bias gradient
  int64_t P, N;
  int C, act;
  int lanes, rows;             // columns (N > 1): threads along a channel's batch items, channels per block
  int64_t tiles;               // batch tiles of lanes·V items
};

template <int V>
__device__ __forceinline__ void act_grad_vec(const ActGradArgs& a, int64_t i, float (&g)[V]) {
  if (a.gy.bf16)
    load_bf16<V>(a.gy.p, i, g);
  else
    load_f32<V>(a.gy.p, i, g);
  if (a.z) {
    float z[V];
    load_bf16<V>(a.z, i, z);
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] *= act_slope(z[e], a.act);
  }
  if (a.gz.p) store_vec<V>(a.gz, i, g);
}

// Token rows (N = 1): a block takes 32·V channels of every 8·gridDim.y-th
// group of rows; a thread the same V channels of its rows.
template <int V>
__global__ void __launch_bounds__(256) act_grad_row_kernel(const ActGradArgs a) {
  __shared__ float s[8][32 * V];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * V;
  float acc[V] = {};
  if (c < a.C)
    for (int64_t p = blockIdx.y * 8 + q; p < a.P; p += gridDim.y * 8) {
      float g[V];
      act_grad_vec<V>(a, p * a.C + c, g);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += g[e];
    }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < V; ++e) s[q][lane * V + e] = acc[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * V; i += 256) {
    const int ch = blockIdx.x * 32 * V + i;
    if (ch < a.C) {
      float t = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) t += s[r][i];
      a.part[static_cast<int64_t>(blockIdx.y) * a.C + ch] = t;
    }
  }
}

// Batch columns (N > 1): a block takes `rows` channels of every gridDim.y-th
// (position, batch tile); a thread V batch items of one channel.
template <int V>
__global__ void __launch_bounds__(256) act_grad_tile_kernel(const ActGradArgs a) {
  __shared__ float s[256];
  const int r = threadIdx.x / a.lanes, l = threadIdx.x % a.lanes;
  const int c = blockIdx.x * a.rows + r;
  const bool act = r < a.rows && c < a.C;
  float acc = 0.f;
  for (int64_t t = blockIdx.y; t < a.P * a.tiles; t += gridDim.y) {
    const int64_t p = t / a.tiles, n = ((t % a.tiles) * a.lanes + l) * V;
    if (act && n < a.N) {
      float g[V];
      act_grad_vec<V>(a, (p * a.C + c) * a.N + n, g);
#pragma unroll
      for (int e = 0; e < V; ++e) acc += g[e];
    }
  }
  if (!a.part) return;
  s[threadIdx.x] = acc;
  __syncthreads();
  if (act && l == 0) {
    float t = 0.f;
    for (int i = 0; i < a.lanes; ++i) t += s[r * a.lanes + i];
    a.part[static_cast<int64_t>(blockIdx.y) * a.C + c] = t;
  }
}

}  // namespace mqv
