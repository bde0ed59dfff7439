// Dense product with bias, activation and residual in its epilogue, and its
// gradients (bf16 operands, fp32 accumulation on the matrix cores).
//
// Pages: "Mixtral" study notes, nn.Linear of MixtralMoE (the router) and of
// the projections around the experts.
//
//   y = act(x w^T + bias) + residual
//   dpre = dy act'(pre),  dx = dpre w,  dw = dpre^T x,  dbias = sum_m dpre
//
// All three products are out[r][c] = sum_t P(r, t) Q(c, t); an operand is
// stored with its contraction index contiguous ([r][t]) or as the slow index
// ([t][r], dx: Q = w; dw: P = dpre, Q = x).
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 32, kPad = 8;

// One operand's tile slice (64 rows x 32 of the contraction) into LDS [row][t].
template <bool SLOW>
__device__ __forceinline__ void load_slice(const uint16_t* __restrict__ p, int64_t ld, int r0, int rows, int t0,
                                           int len, uint16_t (*lds)[kStep + kPad]) {
  const int i = threadIdx.x;
  if constexpr (!SLOW) {
    const int r = i >> 2, t = t0 + (i & 3) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r0 + r < rows && t < len) v = *reinterpret_cast<const uint4*>(p + (int64_t)(r0 + r) * ld + t);
    *reinterpret_cast<uint4*>(&lds[r][(i & 3) * 8]) = v;
  } else {
    const int t = i >> 3, r = (i & 7) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t0 + t < len && r0 + r < rows) v = *reinterpret_cast<const uint4*>(p + (int64_t)(t0 + t) * ld + r0 + r);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 8; ++q) lds[r + q][t] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
  }
}

template <bool PSLOW, bool QSLOW>
__global__ __launch_bounds__(256) void linear_tile_kernel(const uint16_t* __restrict__ P, int64_t ldp,
                                                          const uint16_t* __restrict__ Q, int64_t ldq, int rows,
                                                          int cols, int len, int col_tiles, const Epilogue ep) {
  __shared__ __attribute__((aligned(16))) uint16_t ps[kTile][kStep + kPad];
  __shared__ __attribute__((aligned(16))) uint16_t qs[kTile][kStep + kPad];
  const int r0 = (blockIdx.x / col_tiles) * kTile, c0 = (blockIdx.x % col_tiles) * kTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fi = lane & 31, fg = lane >> 5;
  const int wr = (wave >> 1) * 32, wc = (wave & 1) * 32;
  f32x16_t acc = {};
  for (int t = 0; t < len; t += kStep) {
    load_slice<PSLOW>(P, ldp, r0, rows, t, len, ps);
    load_slice<QSLOW>(Q, ldq, c0, cols, t, len, qs);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStep / 16; ++s) {
      const uint4 a = *reinterpret_cast<const uint4*>(&qs[wc + fi][s * 16 + fg * 8]);
      const uint4 b = *reinterpret_cast<const uint4*>(&ps[wr + fi][s * 16 + fg * 8]);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), acc, 0, 0, 0);
    }
    __syncthreads();
  }
  const int r = r0 + wr + fi;
  if (r >= rows) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = c0 + wc + q * 8 + fg * 4;
    if (c < cols) ep.store4(r, c, cols, make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
  }
}

template <bool PSLOW, bool QSLOW>
hipError_t launch_product(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t ldq, int rows, int cols,
                          int len, const Epilogue& ep, hipStream_t st) {
  const int rt = (rows + kTile - 1) / kTile, ct = (cols + kTile - 1) / kTile;
  hipLaunchKernelGGL((linear_tile_kernel<PSLOW, QSLOW>), dim3((unsigned)((int64_t)rt * ct)), dim3(256), 0, st, P,
                     ldp, Q, ldq, rows, cols, len, ct, ep);
  return hipGetLastError();
}

// ---- gradient at the pre-activation ----

constexpr int kPrepCols = 256;      // columns per workgroup, 8 to a lane
constexpr int kPrepRows = 256;      // rows per workgroup: one row of column sums comes of them

// dpre = dy act'(pre) in bf16 (unless NULL), and the column sums of its fp32
// values over the workgroup's rows into part[chunk][N] (unless NULL).
// HBM-bound: reads dy and pre, writes dpre, once each.
template <bool F32, bool ACT>
__global__ __launch_bounds__(256) void dpre_kernel(const void* __restrict__ dy, const uint16_t* __restrict__ pre,
                                                   int act, int M, int N, int col_blocks,
                                                   uint16_t* __restrict__ dpre, float* __restrict__ part) {
  __shared__ float sums[8][kPrepCols];
  const int chunk = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int cl = (threadIdx.x & 31) * 8, rl = threadIdx.x >> 5;
  const int c = cb * kPrepCols + cl;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int r_end = min(M, (chunk + 1) * kPrepRows);
  if (c < N) {
    for (int r = chunk * kPrepRows + rl; r < r_end; r += 8) {
      const int64_t at = (int64_t)r * N + c;
      float v[8];
      if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(dy) + at);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(dy) + at), v);
      }
      if constexpr (ACT) {
        float p[8];
        unpack8(*reinterpret_cast<const uint4*>(pre + at), p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= act_grad(p[i], act);
      }
      if (dpre != nullptr) *reinterpret_cast<uint4*>(dpre + at) = pack8(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[rl][cl + i] = acc[i];
  __syncthreads();
  const int col = cb * kPrepCols + threadIdx.x;
  if (col < N) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sums[i][threadIdx.x];
    part[(int64_t)chunk * N + col] = s;
  }
}

// dbias[c] = the sum of part[.][c], in chunk order.
__global__ __launch_bounds__(256) void dbias_kernel(const float* __restrict__ part, int chunks, int N,
                                                    float* __restrict__ dbias) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= N) return;
  float s = 0.f;
  for (int i = 0; i < chunks; ++i) s += part[(int64_t)i * N + c];
  dbias[c] = s;
}

int prep_chunks(const moe_linear_t& l) { return (l.M + kPrepRows - 1) / kPrepRows; }
// dpre has bf16 values of its own unless dy already is what the products read.
bool dpre_copied(const moe_linear_t& l) { return l.act != MOE_ACT_NONE || l.y_dtype == MOE_F32; }

size_t round256(size_t v) { return (v + 255) / 256 * 256; }
size_t dpre_bytes(const moe_linear_t& l) { return dpre_copied(l) ? round256((size_t)l.M * l.N * 2) : 0; }

}  // namespace

size_t linear_workspace_bytes(const moe_linear_t&) { return 0; }

size_t linear_backward_workspace_bytes(const moe_linear_t& l) {
  return dpre_bytes(l) + round256((size_t)prep_chunks(l) * l.N * 4);
}

hipError_t launch_linear(const moe_linear_t& l, const uint16_t* x, const uint16_t* w, const float* bias,
                         const void* residual, void* y, uint16_t* pre, void* workspace, hipStream_t st) {
  (void)workspace;
  const Epilogue ep{bias, residual, y, pre, l.act, l.y_dtype == MOE_F32};
  return launch_product<false, false>(x, l.K, w, l.K, l.M, l.N, l.K, ep, st);
}

hipError_t launch_linear_backward(const moe_linear_t& l, const void* dy, const uint16_t* pre, const uint16_t* x,
                                  const uint16_t* w, uint16_t* dx, uint16_t* dw, float* dbias, void* workspace,
                                  hipStream_t st) {
  uint16_t* copy = dpre_copied(l) && (dx != nullptr || dw != nullptr) ? static_cast<uint16_t*>(workspace) : nullptr;
  float* part = dbias != nullptr ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dpre_bytes(l)) : nullptr;
  hipError_t e = hipSuccess;
  if (copy != nullptr || part != nullptr) {
    const int cbs = (l.N + kPrepCols - 1) / kPrepCols;
    const dim3 grid((unsigned)((int64_t)cbs * prep_chunks(l)));
    const bool f32 = l.y_dtype == MOE_F32, act = l.act != MOE_ACT_NONE;
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, dy, pre, l.act, l.M, l.N, cbs, copy, part);
      return hipGetLastError();
    };
    e = f32 ? (act ? run(dpre_kernel<true, true>) : run(dpre_kernel<true, false>))
            : (act ? run(dpre_kernel<false, true>) : run(dpre_kernel<false, false>));
  }
  if (e == hipSuccess && dbias != nullptr) {
    hipLaunchKernelGGL(dbias_kernel, dim3((l.N + 255) / 256), dim3(256), 0, st, part, prep_chunks(l), l.N, dbias);
    e = hipGetLastError();
  }
  const uint16_t* d = copy != nullptr ? copy : static_cast<const uint16_t*>(dy);
  if (e == hipSuccess && dx != nullptr)
    e = launch_product<false, true>(d, l.N, w, l.K, l.M, l.K, l.N, Epilogue{nullptr, nullptr, dx, nullptr, 0, false}, st);
  if (e == hipSuccess && dw != nullptr)
    e = launch_product<true, true>(d, l.N, x, l.K, l.N, l.K, l.M, Epilogue{nullptr, nullptr, dw, nullptr, 0, false}, st);
  return e;
}

}  // namespace moe
