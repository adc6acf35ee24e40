// What the norm and linear kernels share: tensors of fp32 or bfloat16 (chosen
// at run time, the branch outside the element loops), read and written in
// vectors of V elements.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "mqv_ptx.cuh"

namespace mqv {

// A [P][C][N] tensor of either type.
struct TensorIn {
  const void* p;
  int bf16;
};
struct TensorOut {
  void* p;
  int bf16;
};

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// Two fp32 -> packed bf16 (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two floats in a 64-bit register, and operations on both at once.
using pair_t = unsigned long long;

__device__ __forceinline__ pair_t pair(float lo, float hi) {
  pair_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo(pair_t a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float hi(pair_t a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
  pair_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
  pair_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
  pair_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// V consecutive elements at element offset i; V·size bytes aligned.
template <int V>
__device__ __forceinline__ void load_f32(const void* p, int64_t i, float (&v)[V]) {
  const float* f = static_cast<const float*>(p) + i;
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(f) + q);
      v[4 * q] = t.x;
      v[4 * q + 1] = t.y;
      v[4 * q + 2] = t.z;
      v[4 * q + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = __ldg(f + q);
  }
}

// The same from memory that a kernel still running at this one's start wrote:
// not through the read-only path.
template <int V>
__device__ __forceinline__ void load_cg(const float* f, float (&v)[V]) {
  if constexpr (V == 4) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(f));
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = __ldcg(f + q);
  }
}

template <int V>
__device__ __forceinline__ void load_bf16(const void* p, int64_t i, float (&v)[V]) {
  const uint16_t* h = static_cast<const uint16_t*>(p) + i;
  if constexpr (V == 8) {
    const uint4 t = __ldg(reinterpret_cast<const uint4*>(h));
    v[0] = bf16_lo(t.x), v[1] = bf16_hi(t.x), v[2] = bf16_lo(t.y), v[3] = bf16_hi(t.y);
    v[4] = bf16_lo(t.z), v[5] = bf16_hi(t.z), v[6] = bf16_lo(t.w), v[7] = bf16_hi(t.w);
  } else if constexpr (V == 4) {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(h));
    v[0] = bf16_lo(t.x), v[1] = bf16_hi(t.x), v[2] = bf16_lo(t.y), v[3] = bf16_hi(t.y);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = __uint_as_float(static_cast<uint32_t>(__ldg(h + q)) << 16);
  }
}

template <int V>
__device__ __forceinline__ void store_vec(const TensorOut& t, int64_t i, const float (&v)[V]) {
  if (t.bf16) {
    uint16_t* h = static_cast<uint16_t*>(t.p) + i;
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(h) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                pack_bf16(v[6], v[7]));
    else if constexpr (V == 4)
      *reinterpret_cast<uint2*>(h) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    else {
#pragma unroll
      for (int q = 0; q < V; ++q) h[q] = __bfloat16_as_ushort(__float2bfloat16_rn(v[q]));
    }
  } else {
    float* f = static_cast<float*>(t.p) + i;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q)
        reinterpret_cast<float4*>(f)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    } else {
#pragma unroll
      for (int q = 0; q < V; ++q) f[q] = v[q];
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of a parameter gradient's partial rows, part[b][i] for b < rows, in
// the order of b within each of 32 fixed parts: out0 takes i < n, out1 (which
// may be null) the n after them.  A block of 1024 sums 32 columns.  Launched
// as a programmatic dependent of the kernel that writes the rows.
__global__ void __launch_bounds__(1024)
column_sum_kernel(const float* __restrict__ part, int rows, int64_t n, int pairs, float* __restrict__ out0,
                  float* __restrict__ out1) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane, width = n * pairs;
  pdl_wait_prerequisite();
  float a = 0.f;
  if (i < width)
#pragma unroll 4
    for (int b = q; b < rows; b += 32) a += __ldcg(part + b * width + i);
  s[q][lane] = a;
  __syncthreads();
  // warp q adds column q's 32 parts
  const float t = warp_sum(s[lane][q]);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + q;
  if (lane == 0 && c < width) (c < n ? out0 + c : out1 + (c - n))[0] = t;
}

}  // namespace mqv
