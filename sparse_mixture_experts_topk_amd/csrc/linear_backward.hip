// Gradients of the dense product.
//
//   dpre = dy act'(pre),  dx = dpre w,  dw = dpre^T x,  dbias = sum_m dpre
//
// Both products are tiles (linear_tiles.hpp; fp32 operands: linear_f32.hip) with
// operands as they lie in memory: dx contracts over w's slow index, dw over that
// of dpre and of x.
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_plan.hpp"

namespace moe {
namespace {

// ---- gradient at the pre-activation ----

constexpr int kPrepCols = 256;      // columns per workgroup, 8 to a lane
// Rows per workgroup (one row of column sums comes of them): 256, fewer while that
// leaves under four workgroups per CU (4099 x 256: 18 -> 5 us), 16 at least.  Where one
// workgroup has all rows, its sums are dbias and the second kernel falls away (16 x
// 256 x 4096, whole pass: 15.3 -> 9.0 us; taken up to 64 rows instead, 64 x 4096 x
// 4096 took 41 us for 36).
int prep_rows(const moe_linear_t& l) {
  const int64_t col_blocks = (l.N + kPrepCols - 1) / kPrepCols;
  int rows = 256;
  while (rows > 16 && col_blocks * ((l.M + rows - 1) / rows) < 4 * device_cu_count()) rows /= 2;
  return rows;
}

// dpre = dy act'(pre) in the operands' type (unless NULL), and the column sums of
// its fp32 values over the workgroup's rows into part[chunk][N] (unless NULL).
// F32: dy is fp32; OP32: the operands are (pre and dpre too).  HBM-bound: reads dy
// and pre, writes dpre, once each (8192 x 14336, bf16: 140 us, 5.0 TB/s).
template <bool F32, bool ACT, bool OP32>
__global__ __launch_bounds__(256) void dpre_kernel(const void* __restrict__ dy, const void* __restrict__ pre,
                                                   int act, int M, int N, int col_blocks, int rows,
                                                   void* __restrict__ dpre, float* __restrict__ part) {
  __shared__ float sums[8][kPrepCols];
  const int chunk = blockIdx.x / col_blocks, cb = blockIdx.x % col_blocks;
  const int cl = (threadIdx.x & 31) * 8, rl = threadIdx.x >> 5;
  const int c = cb * kPrepCols + cl;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int r_end = min(M, (chunk + 1) * rows);
  if (c < N) {
    for (int r = chunk * rows + rl; r < r_end; r += 8) {
      const int64_t at = (int64_t)r * N + c;
      float v[8];
      if constexpr (F32) load8f(static_cast<const float*>(dy) + at, v);
      else unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(dy) + at), v);
      if constexpr (ACT) {
        float p[8];
        if constexpr (OP32) load8f(static_cast<const float*>(pre) + at, p);
        else unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pre) + at), p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= act_grad(p[i], act);
      }
      if (dpre != nullptr) {
        if constexpr (OP32) store8f(static_cast<float*>(dpre) + at, v);
        else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dpre) + at) = pack8(v);
      }
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

// dbias[c] = the sum of part[.][c]: 16 lanes to a column, each over every 16th
// chunk, then joined in lane order.
__global__ __launch_bounds__(256) void dbias_kernel(const float* __restrict__ part, int chunks, int N,
                                                    float* __restrict__ dbias) {
  __shared__ float sums[16][16];
  const int cl = threadIdx.x & 15, k = threadIdx.x >> 4, c = blockIdx.x * 16 + cl;
  float s = 0.f;
  if (c < N) {
#pragma unroll 4
    for (int i = k; i < chunks; i += 16) s += part[(int64_t)i * N + c];
  }
  sums[k][cl] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < N) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sums[i][cl];
    dbias[c] = t;
  }
}

int prep_chunks(const moe_linear_t& l) { return (l.M + prep_rows(l) - 1) / prep_rows(l); }
// dpre has values of its own unless dy already is what the products read.
bool dpre_copied(const moe_linear_t& l) { return l.act != MOE_ACT_NONE || l.y_dtype != l.dtype; }

size_t round256(size_t v) { return (v + 255) / 256 * 256; }
size_t dpre_bytes(const moe_linear_t& l) { return dpre_copied(l) ? round256((size_t)l.M * l.N * (l.dtype == MOE_F32 ? 4 : 2)) : 0; }

size_t part_bytes(const moe_linear_t& l) { return round256((size_t)prep_chunks(l) * l.N * 4); }

}  // namespace

size_t linear_backward_workspace_bytes(const moe_linear_t& l) {
  if (l.M == 0) return 0;
  if (l.dtype == MOE_F32) return dpre_bytes(l) + part_bytes(l) + linear_backward_product_bytes_f32(l);
  return dpre_bytes(l) + part_bytes(l) + gradient_workspace(l.M, l.N, l.K);
}

hipError_t launch_linear_backward(const moe_linear_t& l, const void* dy, const void* pre, const void* x,
                                  const void* w, void* dx, void* dw, float* dbias, void* workspace,
                                  hipStream_t st) {
  void* copy = dpre_copied(l) && (dx != nullptr || dw != nullptr) ? workspace : nullptr;
  const bool one_chunk = prep_chunks(l) == 1;
  float* part = dbias == nullptr ? nullptr
                : one_chunk      ? dbias
                                 : reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dpre_bytes(l));
  hipError_t e = hipSuccess;
  if (copy != nullptr || part != nullptr) {
    const int rows = prep_rows(l), cbs = (l.N + kPrepCols - 1) / kPrepCols;
    const dim3 grid((unsigned)((int64_t)cbs * ((l.M + rows - 1) / rows)));
    const bool f32 = l.y_dtype == MOE_F32, act = l.act != MOE_ACT_NONE;
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, dy, pre, l.act, l.M, l.N, cbs, rows, copy, part);
      return hipGetLastError();
    };
    if (l.dtype == MOE_F32) e = act ? run(dpre_kernel<true, true, true>) : run(dpre_kernel<true, false, true>);
    else if (f32) e = act ? run(dpre_kernel<true, true, false>) : run(dpre_kernel<true, false, false>);
    else e = act ? run(dpre_kernel<false, true, false>) : run(dpre_kernel<false, false, false>);
  }
  if (e == hipSuccess && dbias != nullptr && !one_chunk) {
    hipLaunchKernelGGL(dbias_kernel, dim3((l.N + 15) / 16), dim3(256), 0, st, part, prep_chunks(l), l.N, dbias);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const void* d = copy != nullptr ? copy : dy;
  void* partials = static_cast<uint8_t*>(workspace) + dpre_bytes(l) + part_bytes(l);
  if (l.dtype == MOE_F32)
    return launch_linear_products_f32(l, static_cast<const float*>(d), static_cast<const float*>(x),
                                      static_cast<const float*>(w), static_cast<float*>(dx), static_cast<float*>(dw),
                                      partials, st);
  return launch_gradients(static_cast<const uint16_t*>(d), static_cast<const uint16_t*>(x),
                          static_cast<const uint16_t*>(w), static_cast<uint16_t*>(dx), static_cast<uint16_t*>(dw), l.M,
                          l.N, l.K, partials, st);
}

}  // namespace moe
