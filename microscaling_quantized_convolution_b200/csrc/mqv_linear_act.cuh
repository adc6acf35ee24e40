// The linear layer's activations and the epilogue that applies bias,
// activation and residual to fp32 sums.
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
