// Activations and the epilogue of the dense product.
#pragma once
#include "device_common.hpp"
#include "../../include/moe.h"

namespace moe {

// Activations and their slopes.  F32 (fp32 operands): the argument of each exponential
// is carried in two parts, so that no error grows with |p| (silu and gelu (tanh) 8 half
// steps of the value, gelu 16, in either tail, where plain products lose 2 |p|, 2.5 p^2 / 2
// and 8 |2 u| more).  Otherwise it is rounded as it comes: that is a change of p by a few
// half steps, which is what the sum of products behind p is off by itself; here too the
// error is relative to the value.
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }
__device__ __forceinline__ float fast_sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-v)); }

constexpr float kGeluA = 1.5957691216057308f;    // 2 sqrt(2 / pi): 0.5 (1 + tanh(u)) = sigmoid(2 u)
constexpr float kGeluB = 0.044715f;

// Phi(-|p|) of the normal distribution and e = exp(-p^2 / 2): the product of e and
// a polynomial in 1 / (1 + 0.2121 |p|) fitted to Phi(-u) e^(u^2/2) over 0 <= u <=
// 13.6 (these coefficients: relative error 4.4e-8; evaluated in fp32, with a
// reciprocal to 1 ulp, 6.4e-7).  The library's erfc took 96 us for 60 in the
// gradient of 6061 x 8064 values.
template <bool F32>
__device__ __forceinline__ float normal_tail(float p, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.2121f, fabsf(p), 1.0f));
  float q = -0.0648413971f;
  q = fmaf(q, t, 0.243251517f);
  q = fmaf(q, t, -0.256910831f);
  q = fmaf(q, t, 0.274553031f);
  q = fmaf(q, t, -0.0476802252f);
  q = fmaf(q, t, 0.107557312f);
  q = fmaf(q, t, 0.0741440579f);
  q = fmaf(q, t, 0.0853452384f);
  q = fmaf(q, t, 0.0845813006f);
  if constexpr (F32) {
    const float hi = -0.72134751f, lo = -9.62981495e-9f;        // -log2(e) / 2
    const float u = fminf(fabsf(p), 32.0f), sq = u * u;         // 0 from there on
    const float x = sq * hi;
    const float r = fmaf(fmaf(u, u, -sq), hi, fmaf(sq, lo, fmaf(sq, hi, -x)));
    e = __builtin_amdgcn_exp2f(x);
    e = fmaf(e, r * 0.693147182f, e);
  } else {
    e = __builtin_amdgcn_exp2f(p * p * -0.7213475204f);
  }
  return q * t * e;
}

// sigmoid(2 u) and 1 - sigmoid(2 u), u = sqrt(2 / pi) (p + 0.044715 p^3), from 2^-|2 u
// log2(e)| with that exponent in two parts; |p| <= 32 (0 and 1 exactly from there on).
__device__ __forceinline__ void tanh_sigmoids(float p, float& s, float& below) {
  constexpr double kA = 2.302208198144325;                      // 2 sqrt(2 / pi) log2(e)
  constexpr float a = (float)kA, a_lo = (float)(kA - (double)a), b_lo = (float)(0.044715 - (double)kGeluB);
  const float sq = p * p, sq_lo = fmaf(p, p, -sq);
  const float g = fmaf(kGeluB, sq, 1.0f);                       // (1 - g is exact: g >= 1 is a multiple of its own step)
  const float g_lo = fmaf(kGeluB, sq, 1.0f - g) + fmaf(kGeluB, sq_lo, b_lo * sq);
  const float v = p * g, v_lo = fmaf(p, g_lo, fmaf(p, g, -v));
  const float x = v * a, r = fmaf(v_lo, a, fmaf(v, a_lo, fmaf(v, a, -x)));
  float e = __builtin_amdgcn_exp2f(-fabsf(x));
  e = fmaf(e, (x < 0.0f ? r : -r) * 0.693147182f, e);
  const float n = __builtin_amdgcn_rcpf(1.0f + e);
  s = x < 0.0f ? e * n : n;
  below = x < 0.0f ? n : e * n;
}
__device__ __forceinline__ float to_32(float p) { return p < -32.0f ? -32.0f : p > 32.0f ? 32.0f : p; }   // NaN stays

template <int ACT, bool F32 = false>
__device__ __forceinline__ float act_value(float p) {
  if constexpr (ACT == MOE_ACT_RELU) return p < 0.0f ? 0.0f : p;          // NaN stays NaN
  else if constexpr (ACT == MOE_ACT_SILU) return p * (F32 ? sigmoid(p) : fast_sigmoid(p));
  else if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    const float q = normal_tail<F32>(p, e);
    return p * (p < 0.0f ? q : 1.0f - q);
  }
  else if constexpr (ACT == MOE_ACT_GELU_TANH) {
    if constexpr (!F32) return p * fast_sigmoid(kGeluA * (p + kGeluB * p * p * p));
    float s, below;
    tanh_sigmoids(to_32(p), s, below);
    return p * s;
  }
  else return p;
}

template <bool F32>
__device__ __forceinline__ float act_grad(float p, int act) {
  switch (act) {
    case MOE_ACT_RELU: return p > 0.0f ? 1.0f : 0.0f;
    case MOE_ACT_SILU: {
      float s, below;
      if constexpr (F32) {
        sigmoids(p, s, below);
      } else {
        s = fast_sigmoid(p);
        below = 1.0f - s;
      }
      return s * (1.0f + p * below);
    }
    case MOE_ACT_GELU: {
      p = to_32(p);                                      // 0 or 1 exactly from there on; p * p stays finite
      float e;
      const float q = normal_tail<F32>(p, e);
      return fmaf(p * e, 0.3989422804014327f, p < 0.0f ? q : 1.0f - q);
    }
    case MOE_ACT_GELU_TANH: {
      p = to_32(p);
      float s, below;
      if constexpr (F32) {
        tanh_sigmoids(p, s, below);
      } else {
        s = fast_sigmoid(kGeluA * (p + kGeluB * p * p * p));
        below = 1.0f - s;
      }
      return s + p * s * below * kGeluA * (1.0f + 3.0f * kGeluB * p * p);
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

__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8f(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 16 bytes to memory; STREAM: non-temporal, so that a large output does not push
// the operands out of L2.
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), static_cast<u32x4_t*>(p));
  else *static_cast<uint4*>(p) = v;
}

// y = act(acc + bias) + residual, 8 channels of one row at a time (channel
// counts are multiples of 8, so a group of 8 is in or out as a whole).
struct Epilogue {
  const float* bias;
  const void* residual;
  void* y;
  uint16_t* pre;
  int f32;       // y and residual

  template <int ACT, bool STREAM = false>
  __device__ __forceinline__ void store8(int r, int c, int cols, float (&v)[8]) const {
    const int64_t at = (int64_t)r * cols + c;
    float u[8];
    if (bias != nullptr) {
      load8f(bias + c, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
    if (pre != nullptr) store16<STREAM>(pre + at, pack8(v));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value<ACT>(v[i]);
    if (residual != nullptr) {
      if (f32) load8f(static_cast<const float*>(residual) + at, u);
      else unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(residual) + at), u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += u[i];
    }
    if (f32) {
      float* o = static_cast<float*>(y) + at;
      store16<STREAM>(o, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
      store16<STREAM>(o + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
      store16<STREAM>(static_cast<uint16_t*>(y) + at, pack8(v));
    }
  }
};

// fp32 operands (linear_f32.hip).
size_t linear_workspace_bytes_f32(const moe_linear_t& l);
size_t linear_backward_product_bytes_f32(const moe_linear_t& l);
hipError_t launch_linear_f32(const moe_linear_t& l, const float* x, const float* w, const float* bias,
                             const float* residual, float* y, float* pre, void* workspace, hipStream_t st);
hipError_t launch_linear_products_f32(const moe_linear_t& l, const float* dpre, const float* x, const float* w,
                                      float* dx, float* dw, void* partials, hipStream_t st);

// Weight streaming for up to kLinearDecodeRows rows (MI355X, us, 32 rows streamed
// against 33 in tiles: 4096 x 4096 11.1 / 15.6, 14336 x 4096 26.0 / 30.8; 64 rows
// streamed four blocks at a time 34.7 against 31.2).
constexpr int kLinearDecodeRows = 32;
// The part of the output that one workgroup of the stream has.  16 channels of all
// rows, read by 8 wavefronts, one stage in flight each.  Two blocks of 16 rows leave
// LDS for one such workgroup per CU: where there are more channels than one round
// of them takes, 4 wavefronts on 32 channels, two workgroups per CU, share each read
// of x twice.  MI355X, us, wide against narrow: 32 rows of 4096 terms, N 4096 13.3 /
// 11.6, N 6144 14.3 / 18.7, N 14336 25.8 / 35.3; with 16 rows N 12288 21.8 / 19.3, N
// 14336 23.1 / 24.0.  16 wavefronts or two stages in flight gain nothing (16 rows, N
// 4096: 10.2, 9.6 / 9.2).  Few channels are bound by what one CU takes in (its part
// of w and of x): 8 channels of 8 or 4 rows, two stages in flight, where the CUs hold
// that many blocks (16 rows of 4096 terms, N 256: 4.3 / 6.8, N 1024: 5.1 / 7.1; of
// 512 terms, N 512: 3.3 / 3.0).
struct DecodeBlock {
  int rows, channels;
  static DecodeBlock of(const moe_linear_t& l, int cus) {
    const int eights = (l.N + 7) / 8;
    if (eights * ((l.M + 3) / 4) <= cus) return {4, 8};
    if (eights * ((l.M + 7) / 8) <= cus) return {8, 8};
    if (l.M <= 16) return {16, 16};
    return {32, (l.N + 15) / 16 > cus ? 32 : 16};
  }
};
hipError_t launch_linear_decode(const moe_linear_t& l, const DecodeBlock& block, const uint16_t* x, const uint16_t* w,
                                const Epilogue& ep, hipStream_t st);

}  // namespace moe
