// Dense product and its gradients with fp32 operands (v_mfma_f32_16x16x4_f32,
// fp32 accumulation): the formulas of linear.hip and linear_backward.hip, with
// pre and dpre in fp32 too, so nothing is rounded below fp32.
//
// All products are out[r][c] = sum_t P(r, t) Q(c, t); an operand is stored [r][t]
// or, SLOW, [t][r].  A workgroup of 4 wavefronts (2 x 2) computes a tile of
// 32 B x 32 B, each wavefront B x B blocks of 16 x 16.  The contraction advances
// 16 at a time: the next slice is loaded into registers while this one is
// multiplied from LDS.  An LDS row holds the 16 terms of one operand row; lane
// (i, g) reads row i's terms 4 g .. 4 g + 3 at once and instruction s takes term
// 4 g + s of both operands (any order of the terms will do, as long as it is the
// same one).  16-byte chunk c of row r sits at c ^ ((r >> 2) & 3): the 16 rows of
// a read phase cover all banks.  Bound by the fp32 matrix rate (157 TFLOP/s):
// 4096^3 1128 us, 122 TFLOP/s (library 138), its gradients 2596 us; few rows by
// the latency of a short contraction and the join: 16 x 256 x 4096 12.1 us.
// Where the tiles leave CUs idle the contraction is cut into equal runs whose
// fp32 results are summed in order by a second kernel.
#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"

namespace moe {
namespace {

constexpr int kTerms = 16;

struct EpilogueF32 {
  const float* bias;
  const float* residual;
  float* y;
  float* pre;

  template <int ACT>
  __device__ __forceinline__ void store4(int r, int c, int cols, float4 v) const {
    const int64_t at = (int64_t)r * cols + c;
    if (bias != nullptr) {
      const float4 b = *reinterpret_cast<const float4*>(bias + c);
      v.x += b.x; v.y += b.y; v.z += b.z; v.w += b.w;
    }
    if (pre != nullptr) *reinterpret_cast<float4*>(pre + at) = v;
    v = make_float4(act_value<ACT, true>(v.x), act_value<ACT, true>(v.y), act_value<ACT, true>(v.z),
                    act_value<ACT, true>(v.w));
    if (residual != nullptr) {
      const float4 q = *reinterpret_cast<const float4*>(residual + at);
      v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
    }
    *reinterpret_cast<float4*>(y + at) = v;
  }
};

struct ArgsF32 {
  const float* P;
  const float* Q;
  int64_t ldp, ldq;
  int rows, cols, len;
  int col_tiles, run, runs;      // terms of a run, runs per tile
  float* partials;               // [runs][rows][cols] when runs > 1
  EpilogueF32 ep;
};

// This thread's parts of an operand's slice (rows x 16 terms, 16 bytes each).
template <bool SLOW, int ROWS>
struct SliceF32 {
  static constexpr int N = ROWS * kTerms / 4 / 256;
  float4 v[N];

  __device__ __forceinline__ void load(const float* p, int64_t ld, int r0, int rows, int t0, int end) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + 256 * k;
      const int r = r0 + (SLOW ? i % (ROWS / 4) * 4 : i / 4), t = t0 + (SLOW ? i / (ROWS / 4) : i % 4 * 4);
      v[k] = r < rows && t < end
                 ? *reinterpret_cast<const float4*>(SLOW ? p + (int64_t)t * ld + r : p + (int64_t)r * ld + t)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float* lds) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + 256 * k;
      if constexpr (SLOW) {
        const int r = i % (ROWS / 4) * 4, t = i / (ROWS / 4);       // 4 rows r .., one swizzle key
        const int at = (((t >> 2) ^ ((r >> 2) & 3)) << 2) + (t & 3);
        lds[(r + 0) * kTerms + at] = v[k].x;
        lds[(r + 1) * kTerms + at] = v[k].y;
        lds[(r + 2) * kTerms + at] = v[k].z;
        lds[(r + 3) * kTerms + at] = v[k].w;
      } else {
        const int r = i / 4, c = i % 4;
        *reinterpret_cast<float4*>(lds + r * kTerms + ((c ^ ((r >> 2) & 3)) << 2)) = v[k];
      }
    }
  }
};

template <bool PSLOW, bool QSLOW, int ACT, int B>
__global__ __launch_bounds__(256) void linear_f32_kernel(const ArgsF32 a) {
  constexpr int T = 32 * B;
  __shared__ __attribute__((aligned(16))) float ps[2][T * kTerms];
  __shared__ __attribute__((aligned(16))) float qs[2][T * kTerms];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int run = blockIdx.x % a.runs, tile = blockIdx.x / a.runs;
  const int r0 = tile / a.col_tiles * T, c0 = tile % a.col_tiles * T;
  const int t0 = run * a.run, end = min(a.len, t0 + a.run);
  const int wr = (wave >> 1) * 16 * B, wc = (wave & 1) * 16 * B;
  f32x4_t acc[B][B];
#pragma unroll
  for (int x = 0; x < B; ++x)
#pragma unroll
    for (int y = 0; y < B; ++y) acc[x][y] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  SliceF32<PSLOW, T> p;
  SliceF32<QSLOW, T> q;
  p.load(a.P, a.ldp, r0, a.rows, t0, end);
  q.load(a.Q, a.ldq, c0, a.cols, t0, end);
  int stage = 0;
  for (int t = t0; t < end; t += kTerms, stage ^= 1) {
    p.store(ps[stage]);
    q.store(qs[stage]);
    __syncthreads();      // (the other stage's readers were past it at the last barrier)
    if (t + kTerms < end) {
      p.load(a.P, a.ldp, r0, a.rows, t + kTerms, end);
      q.load(a.Q, a.ldq, c0, a.cols, t + kTerms, end);
    }
    float4 fa[B], fb[B];
#pragma unroll
    for (int x = 0; x < B; ++x) {
      const int c = wc + x * 16 + i, r = wr + x * 16 + i;
      fa[x] = *reinterpret_cast<const float4*>(&qs[stage][c * kTerms + ((g ^ ((c >> 2) & 3)) << 2)]);
      fb[x] = *reinterpret_cast<const float4*>(&ps[stage][r * kTerms + ((g ^ ((r >> 2) & 3)) << 2)]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int x = 0; x < B; ++x)
#pragma unroll
        for (int y = 0; y < B; ++y)
          acc[x][y] = __builtin_amdgcn_mfma_f32_16x16x4f32(reinterpret_cast<const float*>(&fa[x])[s],
                                                           reinterpret_cast<const float*>(&fb[y])[s], acc[x][y], 0, 0, 0);
  }
  // lane (i, g): row y 16 + i, columns x 16 + 4 g .. + 3
#pragma unroll
  for (int y = 0; y < B; ++y) {
    const int r = r0 + wr + y * 16 + i;
    if (r >= a.rows) continue;
#pragma unroll
    for (int x = 0; x < B; ++x) {
      const int c = c0 + wc + x * 16 + 4 * g;
      if (c >= a.cols) continue;
      const float4 v = make_float4(acc[x][y][0], acc[x][y][1], acc[x][y][2], acc[x][y][3]);
      if (a.runs > 1) *reinterpret_cast<float4*>(a.partials + ((int64_t)run * a.rows + r) * a.cols + c) = v;
      else a.ep.template store4<ACT>(r, c, a.cols, v);
    }
  }
}

// Sums the runs' results in order and applies the epilogue, 4 columns to a lane.
template <int ACT>
__global__ __launch_bounds__(256) void linear_f32_join_kernel(const ArgsF32 a) {
  const int64_t quad = (int64_t)blockIdx.x * 256 + threadIdx.x, total = (int64_t)a.rows * a.cols;
  if (quad * 4 >= total) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < a.runs; ++s) {
    const float4 p = *reinterpret_cast<const float4*>(a.partials + s * total + quad * 4);
    v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
  }
  a.ep.template store4<ACT>((int)(quad * 4 / a.cols), (int)(quad * 4 % a.cols), a.cols, v);
}

// 128 x 128 tiles where they give every CU one, 64 x 64 otherwise (MI355X, us, large
// against small: 4096^3 1128 / 1239, 2048^3 159 / 158, 512 x 256 x 4096 26.4 / 21.7);
// the contraction in as many runs as give each CU two workgroups, each run of 64
// terms at least, and no more than 64 (16 x 256 x 4096: 64 runs).
struct PlanF32 {
  bool large;
  int row_tiles, col_tiles, run, runs;
  static PlanF32 of(int rows, int cols, int len) {
    PlanF32 p;
    const int64_t cus = device_cu_count();
    p.large = (int64_t)((rows + 127) / 128) * ((cols + 127) / 128) >= cus;
    const int T = p.large ? 128 : 64;
    p.row_tiles = (rows + T - 1) / T;
    p.col_tiles = (cols + T - 1) / T;
    const int64_t tiles = (int64_t)p.row_tiles * p.col_tiles;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(64, 2 * cus / tiles), len / 64));
    p.run = (int)((len + want - 1) / want + kTerms - 1) / kTerms * kTerms;
    p.runs = (len + p.run - 1) / p.run;
    return p;
  }
  size_t workspace(int rows, int cols) const { return runs > 1 ? (size_t)runs * rows * cols * 4 : 0; }
};

template <bool PSLOW, bool QSLOW, int ACT>
hipError_t launch_f32(const float* P, int64_t ldp, const float* Q, int64_t ldq, int rows, int cols, int len,
                      void* partials, const EpilogueF32& ep, hipStream_t st) {
  const PlanF32 p = PlanF32::of(rows, cols, len);
  const ArgsF32 a{P, Q, ldp, ldq, rows, cols, len, p.col_tiles, p.run, p.runs, static_cast<float*>(partials), ep};
  const dim3 grid((unsigned)((int64_t)p.row_tiles * p.col_tiles * p.runs));
  if (p.large) hipLaunchKernelGGL((linear_f32_kernel<PSLOW, QSLOW, ACT, 4>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((linear_f32_kernel<PSLOW, QSLOW, ACT, 2>), grid, dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.runs == 1) return e;
  const int64_t quads = (int64_t)rows * cols / 4;
  hipLaunchKernelGGL(linear_f32_join_kernel<ACT>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

size_t product_bytes(int rows, int cols, int len) { return PlanF32::of(rows, cols, len).workspace(rows, cols); }

}  // namespace

size_t linear_workspace_bytes_f32(const moe_linear_t& l) { return l.M == 0 ? 0 : product_bytes(l.M, l.N, l.K); }

size_t linear_backward_product_bytes_f32(const moe_linear_t& l) {
  return std::max(product_bytes(l.M, l.K, l.N), product_bytes(l.N, l.K, l.M));
}

hipError_t launch_linear_f32(const moe_linear_t& l, const float* x, const float* w, const float* bias,
                             const float* residual, float* y, float* pre, void* workspace, hipStream_t st) {
  const EpilogueF32 ep{bias, residual, y, pre};
  auto run = [&](auto act) {
    return launch_f32<false, false, decltype(act)::value>(x, l.K, w, l.K, l.M, l.N, l.K, workspace, ep, st);
  };
  switch (l.act) {
    case MOE_ACT_RELU: return run(std::integral_constant<int, MOE_ACT_RELU>{});
    case MOE_ACT_SILU: return run(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU: return run(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH: return run(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    default: return run(std::integral_constant<int, MOE_ACT_NONE>{});
  }
}

hipError_t launch_linear_products_f32(const moe_linear_t& l, const float* dpre, const float* x, const float* w,
                                      float* dx, float* dw, void* partials, hipStream_t st) {
  hipError_t e = hipSuccess;
  if (dx != nullptr)
    e = launch_f32<false, true, MOE_ACT_NONE>(dpre, l.N, w, l.K, l.M, l.K, l.N, partials,
                                              EpilogueF32{nullptr, nullptr, dx, nullptr}, st);
  if (e == hipSuccess && dw != nullptr)
    e = launch_f32<true, true, MOE_ACT_NONE>(dpre, l.N, x, l.K, l.N, l.K, l.M, partials,
                                             EpilogueF32{nullptr, nullptr, dw, nullptr}, st);
  return e;
}

}  // namespace moe
