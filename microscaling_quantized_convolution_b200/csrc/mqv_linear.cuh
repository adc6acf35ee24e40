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

// Eight consecutive bfloat16 elements from element i of `src`, which need not
// be aligned: fetch() loads the two aligned vectors around them, value() takes
// them out.  The same i % 8 in all lanes of a warp keeps the selection
// uniform.  Elements at `total` and behind are not read, and come as zeros.
struct Unaligned {
  uint4 a, b;

  __device__ __forceinline__ void fetch(const uint16_t* __restrict__ src, int64_t i, int64_t total) {
    const int64_t i0 = i & ~int64_t{7}, last = (total & ~int64_t{7}) - 8;     // the last whole vector
    if (last < 0) return;
    a = __ldg(reinterpret_cast<const uint4*>(src + min(i0, last)));
    b = __ldg(reinterpret_cast<const uint4*>(src + min(i0 + 8, last)));
  }

  __device__ __forceinline__ uint4 value(const uint16_t* __restrict__ src, int64_t i, int64_t total) const {
    const int sh = static_cast<int>(i & 7);
    if (i - sh + 16 > total) {
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] = i + k < total ? __ldg(src + i + k) : 0;
      return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    uint32_t w0, w1, w2, w3, w4;
    switch (sh >> 1) {
      case 0: w0 = a.x, w1 = a.y, w2 = a.z, w3 = a.w, w4 = b.x; break;
      case 1: w0 = a.y, w1 = a.z, w2 = a.w, w3 = b.x, w4 = b.y; break;
      case 2: w0 = a.z, w1 = a.w, w2 = b.x, w3 = b.y, w4 = b.z; break;
      default: w0 = a.w, w1 = b.x, w2 = b.y, w3 = b.z, w4 = b.w; break;
    }
    if (sh & 1)
      return make_uint4(__funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16), __funnelshift_r(w2, w3, 16),
                        __funnelshift_r(w3, w4, 16));
    return make_uint4(w0, w1, w2, w3);
  }
};

// Rows of `len` elements copied to rows `pitch` apart (a multiple of 8), for
// operands whose own rows do not start on the 16-byte boundaries that a TMA
// load needs.  What lies between len and pitch is never read.  `per` threads
// (a power of two up to a warp) copy a row, four 16-byte vectors each in
// flight.
__global__ void __launch_bounds__(256)
repitch_kernel(const uint16_t* __restrict__ src, uint16_t* __restrict__ dst, int64_t rows, int len, int pitch, int per) {
  const int64_t total = rows * len, step = static_cast<int64_t>(gridDim.x) * (256 / per);
  const int c0 = (threadIdx.x & (per - 1)) * 8, hop = per * 8;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / per) + threadIdx.x / per; r < rows; r += step)
    for (int c = c0; c < pitch; c += 4 * hop) {
      Unaligned v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k * hop < pitch) v[k].fetch(src, r * len + c + k * hop, total);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k * hop < pitch)
          *reinterpret_cast<uint4*>(dst + r * pitch + c + k * hop) = v[k].value(src, r * len + c + k * hop, total);
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

// ------------------------------------------------------------- few tokens
//
// P <= kFewTokens token rows: the weights are read once, `split` warps R rows
// of them, 16 bytes a lane and step and eight steps in flight, against the
// tokens' values from L1; the sums stay in registers.  Bound by the weights'
// bytes and the latency of their loads: one token 4096 -> 4096 12 us from HBM,
// 4096 -> 16384 30 us, 4.4 TB/s (0.69 of the copy rate).  ODD, where rows are
// unaligned: the weights are taken out of the aligned vectors around them, the
// tokens' values come one by one (4095 -> 4095: 24 us).

constexpr int kFewTokens = 4;
constexpr int kFewThreads = 128;

template <int P, int R, bool ODD>
__global__ void __launch_bounds__(kFewThreads)
few_tokens_kernel(const Epilogue e, const uint16_t* __restrict__ w, const uint16_t* __restrict__ x, int cin, int cout,
                  int split) {
  constexpr int U = 8 / R, kWarps = kFewThreads / 32;
  __shared__ float parts[kWarps][R * P];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5, mine = warp & (split - 1);
  const int row = (blockIdx.x * (kWarps / split) + warp / split) * R;
  // behind the last row: that one again
  int64_t at[R];
#pragma unroll
  for (int r = 0; r < R; ++r) at[r] = static_cast<int64_t>(min(row + r, cout - 1)) * cin;
  const int64_t total = static_cast<int64_t>(cout) * cin;
  pair_t acc[R][P];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int p = 0; p < P; ++p) acc[r][p] = 0;
  const int hop = split * 256;
  for (int i0 = (mine * 32 + lane) * 8; i0 < cin; i0 += U * hop) {
    uint4 t[U][R];
    if constexpr (ODD) {
      Unaligned v[U][R];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (i0 + u * hop < cin) v[u][r].fetch(w, at[r] + i0 + u * hop, total);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (i0 + u * hop < cin) t[u][r] = v[u][r].value(w, at[r] + i0 + u * hop, total);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (i0 + u * hop < cin) t[u][r] = __ldcs(reinterpret_cast<const uint4*>(w + at[r] + i0 + u * hop));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * hop, left = cin - i;
      if (left <= 0) break;
      if (ODD && left < 8) {     // the next row's values are not to meet even a zero: they may be NaN
#pragma unroll
        for (int r = 0; r < R; ++r) {
          uint32_t* q = reinterpret_cast<uint32_t*>(&t[u][r]);
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] &= (2 * k < left ? 0xffffu : 0u) | (2 * k + 1 < left ? 0xffff0000u : 0u);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) {
        pair_t q[4];
        if constexpr (ODD) {
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) h[k] = __ldg(x + static_cast<int64_t>(p) * cin + i + (k < left ? k : 0));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            q[k] = pair(2 * k < left ? __uint_as_float(h[2 * k] << 16) : 0.f,
                        2 * k + 1 < left ? __uint_as_float(h[2 * k + 1] << 16) : 0.f);
        } else {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(p) * cin + i));
          q[0] = pair(bf16_lo(v.x), bf16_hi(v.x));
          q[1] = pair(bf16_lo(v.y), bf16_hi(v.y));
          q[2] = pair(bf16_lo(v.z), bf16_hi(v.z));
          q[3] = pair(bf16_lo(v.w), bf16_hi(v.w));
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][p] = fma2(q[0], pair(bf16_lo(t[u][r].x), bf16_hi(t[u][r].x)), acc[r][p]);
          acc[r][p] = fma2(q[1], pair(bf16_lo(t[u][r].y), bf16_hi(t[u][r].y)), acc[r][p]);
          acc[r][p] = fma2(q[2], pair(bf16_lo(t[u][r].z), bf16_hi(t[u][r].z)), acc[r][p]);
          acc[r][p] = fma2(q[3], pair(bf16_lo(t[u][r].w), bf16_hi(t[u][r].w)), acc[r][p]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float v = warp_sum(lo(acc[r][p]) + hi(acc[r][p]));
      if (lane == 0) parts[warp][r * P + p] = v;
    }
  __syncthreads();
  if (mine == 0 && lane < R * P && row + lane / P < cout) {
    float v[1] = {parts[warp][lane]};
    for (int k = 1; k < split; ++k) v[0] += parts[warp + k][lane];
    const int r = row + lane / P;
    epilogue_store<1>(e, static_cast<int64_t>(lane % P) * cout + r, r, r, v);
  }
}

// --------------------------------------- gradient of activation and bias

struct ActGradArgs {
  TensorIn gy;
  const void* z;               // bf16
  TensorOut gz;                // null: not written
  float* part;                 // [gridDim.y·tiles][C]; null: no bias gradient
  int64_t P, N;
  int C;
  int lanes, rows, tiles;      // N > 1: threads along a channel's batch items, channels per block, batch tiles
};

// gz = gy·act'(z) of the vectors at `at`, at + hop, ... (`count` of them), R of
// them loaded before the first is used; their sums by element into acc.  Two
// vectors at four blocks an SM (8187 x 4096, GELU: 37 us on the device) beat
// four at two (42 us).
template <int V, int ACT, bool GB>
__device__ __forceinline__ void act_grad_run(const ActGradArgs& a, int64_t at, int64_t hop, int count, float (&acc)[V]) {
  constexpr int R = V == 1 ? 4 : 2;
  for (int i = 0; i < count; i += R, at += R * hop) {
    float g[R][V], z[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // past the end: the first vector again, its values not used
      const int64_t o = i + r < count ? at + r * hop : at;
      if constexpr (GB)
        load_bf16<V>(a.gy.p, o, g[r]);
      else
        load_f32<V>(a.gy.p, o, g[r]);
      if constexpr (ACT != kActNone) load_bf16<V>(a.z, o, z[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (i + r >= count) break;
      if constexpr (ACT == kActRelu) {
        // selected, not multiplied: where the unit is off, a gradient that
        // overflowed to infinity is dropped like any other
#pragma unroll
        for (int e = 0; e < V; ++e) g[r][e] = z[r][e] > 0.f ? g[r][e] : 0.f;
      } else if constexpr (ACT != kActNone) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const pair_t s = slope_pair<ACT>(pair(z[r][e], e + 1 < V ? z[r][e + 1] : 0.f));
          g[r][e] *= lo(s);
          if (e + 1 < V) g[r][e + 1] *= hi(s);
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += g[r][e];
      if (a.gz.p) store_vec<V>(a.gz, at + r * hop, g[r]);
    }
  }
}

// TOKENS (N = 1): a block of eight warps takes 32·V channels of every
// 8·gridDim.y-th group of rows; a thread the same V channels of its rows.
// Otherwise a block takes `rows` channels and one batch tile of every
// gridDim.y-th position; a thread V batch items of one channel.
template <int V, int ACT, bool TOKENS>
__global__ void __launch_bounds__(256, 4) act_grad_kernel(const ActGradArgs a) {
  __shared__ float s[TOKENS ? 8 * 32 * V : 256];
  float acc[V] = {};
  int64_t at, hop;
  int64_t count;
  int c, r = 0, l = 0;
  int row = blockIdx.y;
  if constexpr (TOKENS) {
    l = threadIdx.x & 31;
    r = threadIdx.x >> 5;
    c = (blockIdx.x * 32 + l) * V;
    const int64_t p = blockIdx.y * 8 + r;
    at = p * a.C + c;
    hop = static_cast<int64_t>(gridDim.y) * 8 * a.C;
    count = c < a.C && p < a.P ? (a.P - p + gridDim.y * 8 - 1) / (gridDim.y * 8) : 0;
  } else {
    r = threadIdx.x / a.lanes;
    l = threadIdx.x - r * a.lanes;
    const int block = blockIdx.x / a.tiles, tile = blockIdx.x - block * a.tiles;
    c = block * a.rows + r;
    row = row * a.tiles + tile;
    const int64_t n = (static_cast<int64_t>(tile) * a.lanes + l) * V;
    at = (blockIdx.y * static_cast<int64_t>(a.C) + c) * a.N + n;
    hop = static_cast<int64_t>(gridDim.y) * a.C * a.N;
    count = r < a.rows && c < a.C && n < a.N && blockIdx.y < a.P ? (a.P - blockIdx.y + gridDim.y - 1) / gridDim.y : 0;
  }
  if (a.gy.bf16)
    act_grad_run<V, ACT, true>(a, at, hop, static_cast<int>(count), acc);
  else
    act_grad_run<V, ACT, false>(a, at, hop, static_cast<int>(count), acc);
  pdl_launch_dependents();
  if (!a.part) return;
  if constexpr (TOKENS) {
#pragma unroll
    for (int e = 0; e < V; ++e) s[r * 32 * V + l * V + e] = acc[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
      const int ch = blockIdx.x * 32 * V + i;
      if (ch < a.C) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += s[k * 32 * V + i];
        a.part[static_cast<int64_t>(row) * a.C + ch] = t;
      }
    }
  } else {
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) t += acc[e];
    s[threadIdx.x] = t;
    __syncthreads();
    if (r < a.rows && c < a.C && l == 0) {
      t = 0.f;
      for (int i = 0; i < a.lanes; ++i) t += s[r * a.lanes + i];
      a.part[static_cast<int64_t>(row) * a.C + c] = t;
    }
  }
}

}  // namespace mqv
