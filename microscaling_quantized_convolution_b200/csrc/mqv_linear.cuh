// The matrix product over the channels of a [P][C][N] tensor, with bias,
// activation and residual in its epilogue, and its gradients:
//   z[co][j] = sum_ci w[co][ci]·x[ci][j] + bias[co],  y = act(z) + residual,
//   gz = gy·act'(z), gbias[co] = sum_j gz[co][j],
//   gx[ci][j] = sum_co w[co][ci]·gz[co][j],  gw[co][ci] = sum_j gz[co][j]·x[ci][j],
// where j runs over the columns (p, n) of the tensors.  Operands are
// bfloat16, sums fp32.
#pragma once

#include "mqv_linear_act.cuh"
#include "mqv_ptx.cuh"

namespace mqv {

// ----------------------------------------------------- around the product

// Rows of `len` elements copied to rows `pitch` apart (a multiple of 8), for
// operands whose own rows do not start on the 16-byte boundaries that a TMA
// load needs.  What lies between len and pitch is never read.  A thread
// writes one 16-byte vector, from the two aligned source vectors around it.
__global__ void __launch_bounds__(256)
repitch_kernel(const uint16_t* __restrict__ src, uint16_t* __restrict__ dst, int64_t rows, int len, int pitch) {
  const int per = pitch / 8;
  const int64_t total = rows * len, units = rows * per;
  for (int64_t u = blockIdx.x * int64_t{256} + threadIdx.x; u < units; u += gridDim.x * int64_t{256}) {
    const int64_t r = u / per;
    const int c = static_cast<int>(u - r * per) * 8;
    const int64_t i = r * len + c, i0 = i & ~int64_t{7};
    const int sh = static_cast<int>(i - i0);
    uint4 out;
    if (i0 + 16 <= total) {
      const uint4 lo = __ldg(reinterpret_cast<const uint4*>(src + i0));
      const uint4 hi = sh ? __ldg(reinterpret_cast<const uint4*>(src + i0 + 8)) : lo;
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {      // words of the 8 elements from sh on
          if (j == (sh >> 1) + k) a = w[j];
          if (j == (sh >> 1) + k + 1) b = w[j];
        }
        v[k] = (sh & 1) ? __funnelshift_r(a, b, 16) : a;
      }
      out = make_uint4(v[0], v[1], v[2], v[3]);
    } else {
      uint16_t h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = i + k < total ? __ldg(src + i + k) : uint16_t{0};
      out = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    *reinterpret_cast<uint4*>(dst + r * pitch + c) = out;
  }
}

// The sums of a product split along K, part[s][i], with the epilogue: a block
// takes 32·V elements, warp q the splits q, q + 8, ...; the eight parts are
// added in order.  Element i's channel is (i / inner) % channels, as row of
// the tile when the batch is `inner`, as column when inner = 1.  Launched as a
// programmatic dependent of the product.
template <int V>
__global__ void __launch_bounds__(256)
split_sum_kernel(const Epilogue e, const float* __restrict__ part, int splits, int64_t stride, int64_t n,
                 int64_t inner, int64_t channels) {
  __shared__ float s[8][32 * V];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t i = (blockIdx.x * int64_t{32} + lane) * V;
  pdl_wait_prerequisite();
  float v[V] = {};
  if (i < n)
#pragma unroll 4
    for (int k = q; k < splits; k += 8) {
      float t[V];
      load_cg<V>(part + k * stride + i, t);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] += t[j];
    }
#pragma unroll
  for (int j = 0; j < V; ++j) s[q][lane * V + j] = v[j];
  __syncthreads();
  if (q > 0 || i >= n) return;
  const int parts = splits < 8 ? splits : 8;
  for (int r = 1; r < parts; ++r)
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += s[r][lane * V + j];
  const int64_t ch = e.bias ? (i / inner) % channels : 0;
  epilogue_store<V>(e, i, ch, ch, v);
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
  pdl_launch_dependents();
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
  pdl_launch_dependents();
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
