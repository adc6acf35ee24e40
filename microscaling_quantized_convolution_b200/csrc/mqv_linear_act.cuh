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
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ pair_t exp2_pair(pair_t x) { return pair(exp2_approx(lo(x)), exp2_approx(hi(x))); }
__device__ __forceinline__ pair_t rcp_pair(pair_t x) { return pair(rcp_approx(lo(x)), rcp_approx(hi(x))); }
__device__ __forceinline__ pair_t both(float x) { return pair(x, x); }

// Phi(z), the normal distribution function, and exp(-z^2 / 2), of two values.
// erf by Hastings' approximation (Abramowitz and Stegun 7.1.26): with t =
// 1 / (1 + 0.3275911·x), x = |z| / sqrt 2, 1 - erf(x) = t·poly4(t)·exp(-x^2)
// within 1.5e-7, 0.75e-7 of Phi: less than two roundings of 1 + erf.  Two
// special-function operations and a dozen other instructions a value; the
// library's erff costs three times that, more than the products of a tile
// with 1024 channels.
__device__ __forceinline__ pair_t normal_cdf(pair_t z, pair_t* phi) {
  const pair_t x = pair(fabsf(lo(z)), fabsf(hi(z)));
  const pair_t t = rcp_pair(fma2(x, both(0.3275911f * 0.70710678f), both(1.f)));
  pair_t q = fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
  q = fma2(t, q, both(0.5f * 1.421413741f));
  q = fma2(t, q, both(0.5f * -0.284496736f));
  q = fma2(t, q, both(0.5f * 0.254829592f));
  const pair_t e = exp2_pair(mul2(mul2(z, z), both(-0.72134752f)));      // -log2(e) / 2
  *phi = e;
  const pair_t tail = mul2(mul2(t, q), e), body = fma2(tail, both(-1.f), both(1.f));
  return pair(lo(z) < 0.f ? lo(tail) : lo(body), hi(z) < 0.f ? hi(tail) : hi(body));
}

// 1 / (1 + exp(-z)); exp overflows to infinity for z < -88, where the result is 0.
__device__ __forceinline__ pair_t sigmoid(pair_t z) {
  return rcp_pair(add2(exp2_pair(mul2(z, both(-1.44269504f))), both(1.f)));
}

template <int ACT>
__device__ __forceinline__ pair_t act_pair(pair_t z) {
  if constexpr (ACT == kActGelu) {
    pair_t phi;
    return mul2(z, normal_cdf(z, &phi));
  } else if constexpr (ACT == kActSilu) {
    return mul2(z, sigmoid(z));
  } else if constexpr (ACT == kActRelu) {
    return pair(lo(z) < 0.f ? 0.f : lo(z), hi(z) < 0.f ? 0.f : hi(z));   // a NaN stays one
  } else {
    return z;
  }
}

// The slope of GELU or SiLU.
template <int ACT>
__device__ __forceinline__ pair_t slope_pair(pair_t z) {
  static_assert(ACT == kActGelu || ACT == kActSilu, "no slope of its own");
  if constexpr (ACT == kActGelu) {
    pair_t phi;
    const pair_t c = normal_cdf(z, &phi);
    return fma2(mul2(z, both(0.39894228f)), phi, c);
  } else {
    const pair_t s = sigmoid(z);
    return mul2(s, fma2(z, fma2(s, both(-1.f), both(1.f)), both(1.f)));
  }
}

// The activation of K values, its kind tested once.
template <int ACT, int K>
__device__ __forceinline__ void act_all(float (&v)[K]) {
#pragma unroll
  for (int i = 0; i < K; i += 2) {
    const pair_t y = act_pair<ACT>(pair(v[i], i + 1 < K ? v[i + 1] : 0.f));
    v[i] = lo(y);
    if (i + 1 < K) v[i + 1] = hi(y);
  }
}
template <int K>
__device__ __forceinline__ void act_values(float (&v)[K], int act) {
  if (act == kActGelu)
    act_all<kActGelu>(v);
  else if (act == kActSilu)
    act_all<kActSilu>(v);
  else if (act == kActRelu)
    act_all<kActRelu>(v);
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
  act_values(v, e.act);
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
