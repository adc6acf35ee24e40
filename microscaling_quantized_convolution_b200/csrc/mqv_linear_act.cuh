// The linear layer's activations and the epilogue that applies bias,
// activation and residual to fp32 sums.
#pragma once

#include "mqv_layer_common.cuh"

namespace mqv {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3 };

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Phi(z), the normal distribution function, and phi = exp(-z^2 / 2).
// erf by Hastings' approximation (Abramowitz and Stegun 7.1.26): with t =
// 1 / (1 + 0.3275911·x), x = |z| / sqrt 2, 1 - erf(x) = t·poly4(t)·exp(-x^2)
// within 1.5e-7, 0.75e-7 of Phi: less than two roundings of 1 + erf.  Two
// special-function operations and about a dozen multiply-adds a value; the
// library's erff costs three times that, more than the products of a tile
// with 1024 channels.
__device__ __forceinline__ float normal_cdf(float z, float* phi) {
  const float t = __fdividef(1.f, fmaf(fabsf(z), 0.3275911f * 0.70710678f, 1.f));
  float q = fmaf(t, 1.061405429f, -1.453152027f);
  q = fmaf(t, q, 1.421413741f);
  q = fmaf(t, q, -0.284496736f);
  q = fmaf(t, q, 0.254829592f);
  const float e = exp2_approx(z * z * -0.72134752f);       // -log2(e) / 2
  *phi = e;
  const float tail = 0.5f * t * q * e;
  return z < 0.f ? tail : 1.f - tail;
}

// 1 / (1 + exp(-z)); exp overflows to infinity for z < -88, where the result is 0.
__device__ __forceinline__ float sigmoid(float z) {
  return __fdividef(1.f, 1.f + exp2_approx(z * -1.44269504f));
}

__device__ __forceinline__ float act_value(float z, int act) {
  float phi;
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;       // a NaN stays one
    case kActGelu: return z * normal_cdf(z, &phi);
    case kActSilu: return z * sigmoid(z);
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActGelu: {
      float phi;
      const float c = normal_cdf(z, &phi);
      return fmaf(z * 0.39894228f, phi, c);
    }
    case kActSilu: {
      const float s = sigmoid(z);
      return s * fmaf(z, 1.f - s, 1.f);
    }
    default: return 1.f;
  }
}

// The activation of K values, its kind tested once.
template <int K>
__device__ __forceinline__ void act_values(float (&v)[K], int act) {
  if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = act_value(v[i], kActGelu);
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = act_value(v[i], kActSilu);
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = act_value(v[i], kActRelu);
  }
}

// What becomes of a sum: y = act(sum + bias) + residual, z = sum + bias kept.
struct Epilogue {
  TensorOut d, z;              // z.p null: not kept
  const void* residual;        // of d's type; null: none
  const float* bias;           // null: none
  int bias_on_row;             // bias by the tile's row, else by its column
  int act;
  int vec4;                    // 4 consecutive columns are aligned for vector accesses
};

template <int V>
__device__ __forceinline__ void epilogue_store(const Epilogue& e, int64_t off, int64_t row, int64_t col, float (&v)[V]) {
  if (e.bias) {
    if (e.bias_on_row) {
      const float b = __ldg(e.bias + row);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += b;
    } else {
      float b[V];
      load_f32<V>(e.bias, col, b);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += b[i];
    }
  }
  if (e.z.p) store_vec<V>(e.z, off, v);
  if (e.act != kActNone)
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = act_value(v[i], e.act);
  if (e.residual) {
    // a plain load: the residual may be the output buffer itself
    float r[V];
    if (e.d.bf16) {
      if constexpr (V == 4) {
        const uint2 t = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.residual) + off);
        r[0] = bf16_lo(t.x), r[1] = bf16_hi(t.x), r[2] = bf16_lo(t.y), r[3] = bf16_hi(t.y);
      } else {
        r[0] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(e.residual)[off]) << 16);
      }
    } else {
      if constexpr (V == 4) {
        const float4 t = *reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + off);
        r[0] = t.x, r[1] = t.y, r[2] = t.z, r[3] = t.w;
      } else {
        r[0] = static_cast<const float*>(e.residual)[off];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += r[i];
  }
  store_vec<V>(e.d, off, v);
}

// Four columns of one row, `left` of them inside; to the fp32 partial sums
// when `part` is given.
__device__ __forceinline__ void epilogue_store4(const Epilogue& e, float* part, int64_t off, int64_t row, int64_t col,
                                                int64_t left, float (&v)[4]) {
  if (e.vec4) {                  // then `left` is a multiple of 4
    if (part)
      *reinterpret_cast<float4*>(part + off) = make_float4(v[0], v[1], v[2], v[3]);
    else
      epilogue_store<4>(e, off, row, col, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= left) break;
    float s[1] = {v[i]};
    if (part)
      part[off + i] = s[0];
    else
      epilogue_store<1>(e, off + i, row, col + i, s);
  }
}

}  // namespace mqv
