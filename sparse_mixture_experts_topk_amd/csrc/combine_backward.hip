// Gradient of the gate-weighted combine.
//
// Pages: "Mixtral and Mixture-of-Experts, Explained", y = sum_i G(x)_i *
// Expert_i(x), differentiated: with row = slot_to_row[t, s],
//   dy_perm[row]     = w[t, s] * dy[t]          (shared expert: dy[t])
//   dweights[t, s]   = <dy[t], y_perm[row]>     (a dropped slot: 0)
//
// One workgroup per token, one pass: a lane holds 8 elements of dy[t] and
// meets each slot's row with them.  The products of the dot are summed in
// fp64: the terms cancel (a gate gradient is often far below them), the
// kernel is HBM-bound (reads dy and the kept y_perm rows, writes as many
// dy_perm rows), and the fp64 additions hide under the reads (8192 x 4096, bf16,
// k 8 and a shared expert, MI355X: 380 us, 4.6 TB/s of 4.9 that a copy reaches).
#include "device_common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxTokens = 1 << 23;      // per launch

// K slots and S (0 or 1) shared rows.  A dropped slot reads row 0 (present
// whenever T > 0) and is selected away, so that all loads of a step are in
// flight together.
template <bool BF16, int K, int S>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const void* __restrict__ dy, const float* __restrict__ y_perm, const int32_t* __restrict__ slot_to_row,
    const float* __restrict__ gw, int d, int T, int first, void* __restrict__ dy_perm, float* __restrict__ dweights) {
  constexpr int N = K + S;
  __shared__ double part[kWaves][K];
  const int t = first + blockIdx.x;
  int rows[N];
  float g[N];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    rows[j] = slot_to_row[(int64_t)t * K + j];
    g[j] = gw[(int64_t)t * K + j];
  }
  if constexpr (S == 1) {
    rows[K] = slot_to_row[(int64_t)T * K + t];
    g[K] = 1.0f;
  }
  double dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) dot[j] = 0.0;
  for (int c = threadIdx.x * 8; c < d; c += kThreads * 8) {
    float v[8];
    if constexpr (BF16) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(dy) + (int64_t)t * d + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(dy) + (int64_t)t * d + c);
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    if (dweights != nullptr) {
      uint4 y[K][2];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const float* src = y_perm + (int64_t)(rows[j] >= 0 ? rows[j] : 0) * d + c;
        y[j][0] = load_stream16(src);
        y[j][1] = load_stream16(src + 4);
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const uint32_t yw[8] = {y[j][0].x, y[j][0].y, y[j][0].z, y[j][0].w,
                                y[j][1].x, y[j][1].y, y[j][1].z, y[j][1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[j] = fma((double)v[i], (double)__uint_as_float(yw[i]), dot[j]);
      }
    }
    if (dy_perm != nullptr) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (rows[j] < 0) continue;
        if constexpr (BF16) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dy_perm) + (int64_t)rows[j] * d + c) =
              make_uint4(pack_bf16x2(g[j] * v[0], g[j] * v[1]), pack_bf16x2(g[j] * v[2], g[j] * v[3]),
                         pack_bf16x2(g[j] * v[4], g[j] * v[5]), pack_bf16x2(g[j] * v[6], g[j] * v[7]));
        } else {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(dy_perm) + (int64_t)rows[j] * d + c);
          o[0] = make_float4(g[j] * v[0], g[j] * v[1], g[j] * v[2], g[j] * v[3]);
          o[1] = make_float4(g[j] * v[4], g[j] * v[5], g[j] * v[6], g[j] * v[7]);
        }
      }
    }
  }
  if (dweights == nullptr) return;                           // uniform
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) dot[j] += __shfl_xor(dot[j], m);
  }
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int j = 0; j < K; ++j) part[threadIdx.x >> 6][j] = dot[j];
  }
  __syncthreads();
  const int j = threadIdx.x;
  if (j < K) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += part[w][j];
    dweights[(int64_t)t * K + j] = slot_to_row[(int64_t)t * K + j] >= 0 ? (float)sum : 0.0f;
  }
}

template <int K, int S>
hipError_t launch_ks(const moe_shape_t& s, const void* dy, const float* y_perm, const int32_t* slot_to_row,
                     const float* weights, void* dy_perm, float* dweights, hipStream_t st) {
  // a grid has fewer than 2^32 threads: 2^24 tokens take two launches
  for (int first = 0; first < s.T; first += kMaxTokens) {
    const dim3 grid((unsigned)(s.T - first < kMaxTokens ? s.T - first : kMaxTokens));
    if (s.act_dtype == MOE_BF16)
      hipLaunchKernelGGL((combine_backward_kernel<true, K, S>), grid, dim3(kThreads), 0, st, dy, y_perm,
                         slot_to_row, weights, s.d_model, s.T, first, dy_perm, dweights);
    else
      hipLaunchKernelGGL((combine_backward_kernel<false, K, S>), grid, dim3(kThreads), 0, st, dy, y_perm,
                         slot_to_row, weights, s.d_model, s.T, first, dy_perm, dweights);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int S>
hipError_t launch_k(const moe_shape_t& s, const void* dy, const float* y_perm, const int32_t* slot_to_row,
                    const float* weights, void* dy_perm, float* dweights, hipStream_t st) {
  static_assert(kMaxTopK == 8, "one instance per k");
  switch (s.top_k) {
    case 1: return launch_ks<1, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    case 2: return launch_ks<2, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    case 3: return launch_ks<3, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    case 4: return launch_ks<4, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    case 5: return launch_ks<5, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    case 6: return launch_ks<6, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    case 7: return launch_ks<7, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
    default: return launch_ks<8, S>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
  }
}

}  // namespace

hipError_t launch_combine_backward(const moe_shape_t& s, const void* dy, const float* y_perm,
                                   const int32_t* slot_to_row, const float* weights, void* dy_perm,
                                   float* dweights, hipStream_t st) {
  if (s.n_shared != 0) return launch_k<1>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
  return launch_k<0>(s, dy, y_perm, slot_to_row, weights, dy_perm, dweights, st);
}

}  // namespace moe
