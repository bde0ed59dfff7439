// Gradients of the dense product.
//
//   dpre = dy act'(pre),  dx = dpre w,  dw = dpre^T x,  dbias = sum_m dpre
//
// Both products are tiles (linear_tiles.hpp; fp32 operands: linear_f32.hip) with
// operands as they lie in memory: dx contracts over w's slow index, dw over that
// of dpre and of x.
#include <algorithm>

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
  const int64_t workgroups = 4 * device_cu_count();
  int rows = 256;
  while (rows > 16 && col_blocks * ((l.M + rows - 1) / rows) < workgroups) rows /= 2;
  return rows;
}

// dpre = dy act'(pre) in the operands' type (unless NULL), and the column sums of
// its fp32 values over the workgroup's rows into part[chunk][N] (unless NULL).
// F32: dy is fp32; OP32: the operands are (pre and dpre too).  With bf16 operands
// dpre is rounded to bf16, for the matrix cores take both operands in one type: dx and
// dw are then 2.34e-3 of their size from the exact ones, where their own rounding
// alone makes 1.66e-3.  The low half of dpre as a second operand would take that away
// and double the terms of both products (they are 1420 of 1600 us at 8192 x 14336 x
// 4096); fp32 operands keep all of it.  HBM-bound: reads dy and pre, writes dpre, once
// each (8192 x 14336, bf16: 140 us, 5.0 TB/s).
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
        for (int i = 0; i < 8; ++i) v[i] *= act_grad<OP32>(p[i], act);
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

// dpre has values of its own unless dy already is what the products read.
bool dpre_copied(const moe_linear_t& l) { return l.act != MOE_ACT_NONE || l.y_dtype != l.dtype; }

size_t round256(size_t v) { return (v + 255) / 256 * 256; }
size_t dpre_bytes(const moe_linear_t& l) { return dpre_copied(l) ? round256((size_t)l.M * l.N * (l.dtype == MOE_F32 ? 4 : 2)) : 0; }

size_t part_bytes(const moe_linear_t& l, int rows) { return round256((size_t)((l.M + rows - 1) / rows) * l.N * 4); }

// ---- dbias, dx, dw ----

// Column sums of part[chunks][N]: out[c] = the sum of part[.][c], 16 lanes to a
// column, each over every 16th chunk, then joined in lane order.
struct ColumnSums {
  const float* part;
  float* out;                // NULL: none wanted
  int chunks, N;
};
template <int THREADS>
__device__ __forceinline__ void column_sums_workgroup(const ColumnSums& a, float (&sums)[THREADS], int block) {
  constexpr int COLS = THREADS / 16;
  const int cl = threadIdx.x % COLS, k = threadIdx.x / COLS, c = block * COLS + cl;
  float s = 0.f;
  if (c < a.N) {
#pragma unroll 4
    for (int i = k; i < a.chunks; i += 16) s += a.part[(int64_t)i * a.N + c];
  }
  sums[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < COLS && c < a.N) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += sums[i * COLS + cl];
    a.out[c] = v;
  }
}

__global__ __launch_bounds__(256) void dbias_kernel(const ColumnSums a) {
  __shared__ float sums[256];
  column_sums_workgroup<256>(a, sums, blockIdx.x);
}
hipError_t launch_dbias(const ColumnSums& a, hipStream_t st) {
  if (a.out == nullptr) return hipSuccess;
  hipLaunchKernelGGL(dbias_kernel, dim3((a.N + 15) / 16), dim3(256), 0, st, a);
  return hipGetLastError();
}

// dbias on the first bias_blocks (a multiple of 8) workgroups, dx on the next
// dx_blocks, dw on the others: one launch, and dw's workgroups fill the CUs that
// dx's last round of tiles leaves idle.
template <int NS, int WR, int WC, int WA, int WB>
__global__ __launch_bounds__(64 * WR * WC, 1) void linear_gradients_kernel(const ProductArgs dx, const ProductArgs dw,
                                                                           const ColumnSums dbias, int bias_blocks,
                                                                           int dx_blocks) {
  constexpr int THREADS = 64 * WR * WC;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * ProductGeom<NS, WR, WC, WA, WB>::STAGE];
  static_assert(THREADS * 4 <= sizeof(smem), "the column sums fit");
  if ((int)blockIdx.x < bias_blocks) {
    column_sums_workgroup<THREADS>(dbias, *reinterpret_cast<float (*)[THREADS]>(smem), blockIdx.x);
    return;
  }
  const int b = blockIdx.x - bias_blocks;
  if (b < dx_blocks) product_workgroup<false, true, MOE_ACT_NONE, NS, WR, WC, WA, WB>(dx, smem, b, dx_blocks);
  else
    product_workgroup<true, true, MOE_ACT_NONE, NS, WR, WC, WA, WB>(dw, smem, b - dx_blocks,
                                                                    gridDim.x - bias_blocks - dx_blocks);
}

// The joins of two products of one tile shape, a's on the first a_blocks workgroups.
template <int TA, int TB>
__global__ __launch_bounds__(256) void linear_join2_kernel(const ProductArgs a, const ProductArgs b, int a_slots,
                                                           int b_slots, int a_blocks) {
  const int i = blockIdx.x;
  if (i < a_blocks) join_workgroup<MOE_ACT_NONE, TA, TB>(a, a_slots, i);
  else join_workgroup<MOE_ACT_NONE, TA, TB>(b, b_slots, i - a_blocks);
}

// Both products of a backward pass in one launch, with one tile shape: dw's
// workgroups fill the CUs that dx's last round leaves, and a launch is saved.
// Worth kOneLaunch us against each product in its best shape and dbias alone
// (MI355X, 64 x 512 x 512: 12.1 us against 18.3, 300 x 1024 x 2048: 19.0 against
// 26.7, 4099 x 256 x 4096, by the plan 1.9 us above: 55.2 against 59.8; not 509 x
// 4096 x 2048, 3.4 above: 47.7 against 45.8, nor 1024 x 4096 x 4096, 15 above: 100
// against 92.5).
constexpr double kOneLaunch = 2.5;
struct GradientPlan {
  ProductPlans dx, dw;
  int tile = 0;                      // the shape for both
  bool one;                          // launch; otherwise each product has its own shape

  static GradientPlan of(int M, int N, int K) {
    const int64_t cus = plan_cus(device_cu_count());
    GradientPlan g{ProductPlans::of(M, K, N, 1, cus), ProductPlans::of(N, K, M, 2, cus)};
    for (int i = 1; i < 4; ++i)
      if (g.cost(i) < g.cost(g.tile)) g.tile = i;
    g.one = g.cost(g.tile) <= g.dx.least().cost + g.dw.least().cost + kOneLaunch;
    return g;
  }
  double cost(int i) const { return dx.p[i].cost + dw.p[i].cost; }
  // partial tiles: both products', or those of one at a time
  size_t workspace() const {
    const size_t each = std::max(dx.least().workspace, dw.least().workspace);
    return one ? std::max(each, dx.p[tile].workspace + dw.p[tile].workspace) : each;
  }
};

// dx = dpre w, dw = dpre^T x and dbias; any of them may be NULL.
hipError_t launch_gradients(const uint16_t* dpre, const uint16_t* x, const uint16_t* w, uint16_t* dx, uint16_t* dw,
                            const ColumnSums& dbias, int M, int N, int K, void* partials, hipStream_t st) {
  const Epilogue to_dx{nullptr, nullptr, dx, nullptr, false}, to_dw{nullptr, nullptr, dw, nullptr, false};
  const GradientPlan plan = GradientPlan::of(M, N, K);
  if (!plan.one || dx == nullptr || dw == nullptr) {
    hipError_t e = launch_dbias(dbias, st);
    if (e == hipSuccess && dx != nullptr)
      e = launch_product<false, true, MOE_ACT_NONE>(dpre, N, w, K, M, K, N, plan.dx, partials, to_dx, st);
    if (e == hipSuccess && dw != nullptr)
      e = launch_product<true, true, MOE_ACT_NONE>(dpre, N, x, K, N, K, M, plan.dw, partials, to_dw, st);
    return e;
  }
  return with_tile(plan.tile, [&](auto tile) {
    using C = decltype(tile);
    using G = GeomOf<C>;
    const ProductPlan &px = plan.dx.p[plan.tile], &pw = plan.dw.p[plan.tile];
    const ProductArgs a{dpre, w, N, K, M, K, N, px.row_tiles, px.col_tiles, px.split, static_cast<float*>(partials), to_dx};
    const ProductArgs b{dpre, x, N, K, N, K, M, pw.row_tiles, pw.col_tiles, pw.split,
                        reinterpret_cast<float*>(static_cast<uint8_t*>(partials) + px.workspace), to_dw};
    const int cols = G::THREADS / 16, bias_blocks = dbias.out != nullptr ? (N + 8 * cols - 1) / (8 * cols) * 8 : 0;
    hipLaunchKernelGGL((linear_gradients_kernel<C::NS, C::WR, C::WC, C::WA, C::WB>),
                       dim3((unsigned)(bias_blocks + px.grid + pw.grid)), dim3(G::THREADS), 0, st, a, b, dbias,
                       bias_blocks, px.grid);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(px.split || pw.split)) return e;
    const int ja = px.split ? (int)join_blocks_of<C>(px) : 0, jb = pw.split ? (int)join_blocks_of<C>(pw) : 0;
    hipLaunchKernelGGL((linear_join2_kernel<G::TA, G::TB>), dim3((unsigned)(ja + jb)), dim3(256), 0, st, a, b,
                       px.grid / 8, pw.grid / 8, ja);
    return hipGetLastError();
  });
}

}  // namespace

size_t linear_backward_workspace_bytes(const moe_linear_t& l) {
  if (l.M == 0) return 0;
  const size_t prep = dpre_bytes(l) + part_bytes(l, prep_rows(l));
  if (l.dtype == MOE_F32) return prep + linear_backward_product_bytes_f32(l);
  return prep + GradientPlan::of(l.M, l.N, l.K).workspace();
}

hipError_t launch_linear_backward(const moe_linear_t& l, const void* dy, const void* pre, const void* x,
                                  const void* w, void* dx, void* dw, float* dbias, void* workspace,
                                  hipStream_t st) {
  void* copy = dpre_copied(l) && (dx != nullptr || dw != nullptr) ? workspace : nullptr;
  const int rows = prep_rows(l), chunks = (l.M + rows - 1) / rows;
  const bool one_chunk = chunks == 1;
  float* part = dbias == nullptr ? nullptr
                : one_chunk      ? dbias
                                 : reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dpre_bytes(l));
  hipError_t e = hipSuccess;
  if (copy != nullptr || part != nullptr) {
    const int cbs = (l.N + kPrepCols - 1) / kPrepCols;
    const dim3 grid((unsigned)((int64_t)cbs * chunks));
    const bool f32 = l.y_dtype == MOE_F32, act = l.act != MOE_ACT_NONE;
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, dy, pre, l.act, l.M, l.N, cbs, rows, copy, part);
      return hipGetLastError();
    };
    if (l.dtype == MOE_F32) e = act ? run(dpre_kernel<true, true, true>) : run(dpre_kernel<true, false, true>);
    else if (f32) e = act ? run(dpre_kernel<true, true, false>) : run(dpre_kernel<true, false, false>);
    else e = act ? run(dpre_kernel<false, true, false>) : run(dpre_kernel<false, false, false>);
  }
  if (e != hipSuccess) return e;
  const void* d = copy != nullptr ? copy : dy;
  void* partials = static_cast<uint8_t*>(workspace) + dpre_bytes(l) + part_bytes(l, rows);
  const ColumnSums sums{part, one_chunk ? nullptr : dbias, chunks, l.N};
  if (l.dtype == MOE_F32) {
    e = launch_dbias(sums, st);
    if (e != hipSuccess) return e;
    return launch_linear_products_f32(l, static_cast<const float*>(d), static_cast<const float*>(x),
                                      static_cast<const float*>(w), static_cast<float*>(dx), static_cast<float*>(dw),
                                      partials, st);
  }
  return launch_gradients(static_cast<const uint16_t*>(d), static_cast<const uint16_t*>(x),
                          static_cast<const uint16_t*>(w), static_cast<uint16_t*>(dx), static_cast<uint16_t*>(dw), sums,
                          l.M, l.N, l.K, partials, st);
}

}  // namespace moe
