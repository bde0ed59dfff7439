// Activations and the epilogue of the dense product.
#pragma once
#include "device_common.hpp"
#include "../../include/moe.h"

namespace moe {

// exp by the hardware's exp2: about 1 ulp in fp32 plus the rounding of the
// scaled argument, far below the bf16 rounding that follows.
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }
__device__ __forceinline__ float fast_sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-v)); }

constexpr float kGeluA = 1.5957691216057308f;    // 2 sqrt(2 / pi): 0.5 (1 + tanh(u)) = sigmoid(2 u)
constexpr float kGeluB = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float p) {
  if constexpr (ACT == MOE_ACT_RELU) return fmaxf(p, 0.0f);
  else if constexpr (ACT == MOE_ACT_SILU) return p * fast_sigmoid(p);
  else if constexpr (ACT == MOE_ACT_GELU) return 0.5f * p * erfcf(p * -0.7071067811865476f);   // erfc: exact in the left tail
  else if constexpr (ACT == MOE_ACT_GELU_TANH) return p * fast_sigmoid(kGeluA * (p + kGeluB * p * p * p));
  else return p;
}

__device__ __forceinline__ float act_grad(float p, int act) {
  switch (act) {
    case MOE_ACT_RELU: return p > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
      const float s = fast_sigmoid(p);
      return s * (1.0f + p * (1.0f - s));
    }
    case MOE_ACT_GELU:
      p = fminf(fmaxf(p, -32.0f), 32.0f);   // 0 or 1 exactly from there on; p * p stays finite
      return 0.5f * erfcf(p * -0.7071067811865476f) + p * fast_exp(-0.5f * p * p) * 0.3989422804014327f;
    case MOE_ACT_GELU_TANH: {
      p = fminf(fmaxf(p, -32.0f), 32.0f);
      const float s = fast_sigmoid(kGeluA * (p + kGeluB * p * p * p));
      return s + p * s * (1.0f - s) * kGeluA * (1.0f + 3.0f * kGeluB * p * p);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// y = act(acc + bias) + residual, 4 channels of one row at a time (channel
// counts are multiples of 8, so a group of 4 is in or out as a whole).
struct Epilogue {
  const float* bias;
  const void* residual;
  void* y;
  uint16_t* pre;
  bool f32;      // y and residual

  template <int ACT>
  __device__ __forceinline__ void store4(int r, int c, int cols, float4 v) const {
    const int64_t at = (int64_t)r * cols + c;
    if (bias != nullptr) {
      const float4 b = *reinterpret_cast<const float4*>(bias + c);
      v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    if (pre != nullptr) *reinterpret_cast<uint2*>(pre + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    v.x = act_value<ACT>(v.x); v.y = act_value<ACT>(v.y);
    v.z = act_value<ACT>(v.z); v.w = act_value<ACT>(v.w);
    if (f32) {
      if (residual != nullptr) {
        const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(residual) + at);
        v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
      }
      *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = v;
    } else {
      if (residual != nullptr) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(residual) + at);
        v.x += bf16_lo(q.x); v.y += bf16_hi(q.x); v.z += bf16_lo(q.y); v.w += bf16_hi(q.y);
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  }
};

}  // namespace moe
