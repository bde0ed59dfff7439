// Gradient of the permutation: x_perm[row] = x[token of the row], differentiated,
//
//   dx[t] = addend[t] + sum over the kept slots s of token t of dx_perm[slot_to_row[t, s]]
//
// in fp32 in slot order (the shared expert's row last, the addend first), rounded
// once.  A gather, so there are no atomics and the result repeats.  One workgroup per
// token, 16 bytes of every row to a lane, all rows in flight together (a dropped slot
// reads row 0, there whenever there is a token, and is selected away).  addend and dx may
// be the same memory: a lane reads its 16 bytes before it writes them.  HBM-bound.
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"

namespace moe {
namespace {

constexpr int kMaxTokens = 1 << 23;      // per launch: a grid has fewer than 2^32 threads

template <bool BF16> constexpr int kVec = BF16 ? 8 : 4;
template <bool BF16>
__device__ __forceinline__ void unpack(uint4 u, float (&v)[kVec<BF16>]) {
  if constexpr (BF16) {
    unpack8(u, v);
  } else {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
}

template <bool BF16, int K, int S>
__global__ __launch_bounds__(256) void permute_backward_kernel(const void* __restrict__ dx_perm,
                                                               const int32_t* __restrict__ slot_to_row,
                                                               const void* addend, int d, int T, int first, void* dx) {
  constexpr int N = K + S, V = kVec<BF16>;
  const int t = first + blockIdx.x;
  const int64_t row_bytes = (int64_t)d * (BF16 ? 2 : 4);
  int rows[N];
#pragma unroll
  for (int j = 0; j < K; ++j) rows[j] = slot_to_row[(int64_t)t * K + j];
  if constexpr (S == 1) rows[K] = slot_to_row[(int64_t)T * K + t];
  const uint8_t* src = static_cast<const uint8_t*>(dx_perm);
  for (int64_t b = threadIdx.x * 16; b < row_bytes; b += blockDim.x * 16) {
    uint4 r[N];
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = load_stream16(src + (rows[j] >= 0 ? rows[j] : 0) * row_bytes + b);
    float sum[V];
    if (addend != nullptr) {
      unpack<BF16>(load_stream16(static_cast<const uint8_t*>(addend) + t * row_bytes + b), sum);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float v[V];
      unpack<BF16>(r[j], v);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = rows[j] >= 0 ? sum[i] + v[i] : sum[i];
    }
    uint4 o;
    if constexpr (BF16) o = pack8(sum);
    else o = make_uint4(__float_as_uint(sum[0]), __float_as_uint(sum[1]), __float_as_uint(sum[2]), __float_as_uint(sum[3]));
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(dx) + t * row_bytes + b) = o;
  }
}

template <int K, int S>
hipError_t launch_ks(const moe_shape_t& s, const void* dx_perm, const int32_t* slot_to_row, const void* addend,
                     void* dx, hipStream_t st) {
  const bool bf16 = s.act_dtype == MOE_BF16;
  const int lanes = s.d_model * (bf16 ? 2 : 4) / 16;               // of a row
  const dim3 block(lanes >= 256 ? 256 : (lanes + 63) / 64 * 64);
  for (int first = 0; first < s.T; first += kMaxTokens) {
    const dim3 grid((unsigned)std::min(s.T - first, kMaxTokens));
    if (bf16)
      hipLaunchKernelGGL((permute_backward_kernel<true, K, S>), grid, block, 0, st, dx_perm, slot_to_row, addend,
                         s.d_model, s.T, first, dx);
    else
      hipLaunchKernelGGL((permute_backward_kernel<false, K, S>), grid, block, 0, st, dx_perm, slot_to_row, addend,
                         s.d_model, s.T, first, dx);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int S>
hipError_t launch_k(const moe_shape_t& s, const void* dx_perm, const int32_t* slot_to_row, const void* addend, void* dx,
                    hipStream_t st) {
  static_assert(kMaxTopK == 8, "one instance per k");
  switch (s.top_k) {
    case 1: return launch_ks<1, S>(s, dx_perm, slot_to_row, addend, dx, st);
    case 2: return launch_ks<2, S>(s, dx_perm, slot_to_row, addend, dx, st);
    case 3: return launch_ks<3, S>(s, dx_perm, slot_to_row, addend, dx, st);
    case 4: return launch_ks<4, S>(s, dx_perm, slot_to_row, addend, dx, st);
    case 5: return launch_ks<5, S>(s, dx_perm, slot_to_row, addend, dx, st);
    case 6: return launch_ks<6, S>(s, dx_perm, slot_to_row, addend, dx, st);
    case 7: return launch_ks<7, S>(s, dx_perm, slot_to_row, addend, dx, st);
    default: return launch_ks<8, S>(s, dx_perm, slot_to_row, addend, dx, st);
  }
}

}  // namespace

hipError_t launch_permute_backward(const moe_shape_t& s, const void* dx_perm, const int32_t* slot_to_row,
                                   const void* addend, void* dx, hipStream_t st) {
  if (s.n_shared != 0) return launch_k<1>(s, dx_perm, slot_to_row, addend, dx, st);
  return launch_k<0>(s, dx_perm, slot_to_row, addend, dx, st);
}

}  // namespace moe
