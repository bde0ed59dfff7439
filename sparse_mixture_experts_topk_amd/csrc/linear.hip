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
#include <algorithm>

#include "device_common.hpp"
#include "launch.hpp"
#include "linear_tiles.hpp"

namespace moe {
namespace {

// Tile shapes.
struct Big { static constexpr int NS = 2, WR = 4, WC = 2, WA = 4, WB = 8; };     // 256 x 256, 8 wavefronts
struct Mid { static constexpr int NS = 4, WR = 2, WC = 2, WA = 4, WB = 4; };     // 128 x 128, 4 wavefronts
template <class C> using GeomOf = ProductGeom<C::NS, C::WR, C::WC, C::WA, C::WB>;

// Workgroups: one per CU at most, a multiple of the 8 XCDs, and no more than
// give each at least kMinSlices slices of work.
constexpr int kMinSlices = 4;
template <class C>
struct Plan {
  int row_tiles, col_tiles, KT, grid;
  bool split;
  static Plan of(int rows, int cols, int len) {
    using G = GeomOf<C>;
    Plan p;
    p.row_tiles = (rows + G::TB - 1) / G::TB;
    p.col_tiles = (cols + G::TA - 1) / G::TA;
    p.KT = (len + 63) / 64;
    const int64_t work = (int64_t)p.row_tiles * p.col_tiles * p.KT;
    const int64_t cus = std::min<int64_t>(device_cu_count(), kMaxPersistentGroups) / 8 * 8;
    p.grid = (int)std::max<int64_t>(8, std::min<int64_t>(cus, work / kMinSlices / 8 * 8));
    p.split = false;
    for (int x = 0; x < 8; ++x) {
      const TileSplit s = TileSplit::of(p.row_tiles * p.col_tiles, x, p.grid / 8, p.KT);
      p.split |= s.tail > 0 && !s.whole_tail;
    }
    return p;
  }
  size_t workspace() const { return split ? (size_t)grid * 2 * GeomOf<C>::PARTIAL * 4 : 0; }
};

template <bool PSLOW, bool QSLOW, int ACT, class C>
hipError_t launch_cfg(ProductArgs a, hipStream_t st) {
  using G = GeomOf<C>;
  const Plan<C> p = Plan<C>::of(a.rows, a.cols, a.len);
  a.row_tiles = p.row_tiles;
  a.col_tiles = p.col_tiles;
  hipLaunchKernelGGL((linear_product_kernel<PSLOW, QSLOW, ACT, C::NS, C::WR, C::WC, C::WA, C::WB>),
                     dim3((unsigned)p.grid), dim3(G::THREADS), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.split) return e;
  hipLaunchKernelGGL((linear_join_kernel<ACT, G::TA, G::TB>), dim3((unsigned)(p.grid * (G::TB / 32))), dim3(256), 0,
                     st, a, p.grid / 8, p.KT);
  return hipGetLastError();
}

bool use_big(int rows, int cols, int len) {
  (void)len;
  return (int64_t)((rows + 255) / 256) * ((cols + 255) / 256) >= 192;
}

size_t product_workspace(int rows, int cols, int len) {
  return use_big(rows, cols, len) ? Plan<Big>::of(rows, cols, len).workspace()
                                  : Plan<Mid>::of(rows, cols, len).workspace();
}

template <bool PSLOW, bool QSLOW, int ACT>
hipError_t launch_product(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t ldq, int rows, int cols,
                          int len, void* partials, const Epilogue& ep, hipStream_t st) {
  ProductArgs a{P, Q, ldp, ldq, rows, cols, len, 0, 0, static_cast<float*>(partials), ep};
  if (use_big(rows, cols, len)) return launch_cfg<PSLOW, QSLOW, ACT, Big>(a, st);
  return launch_cfg<PSLOW, QSLOW, ACT, Mid>(a, st);
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

size_t part_bytes(const moe_linear_t& l) { return round256((size_t)prep_chunks(l) * l.N * 4); }

}  // namespace

size_t linear_workspace_bytes(const moe_linear_t& l) { 
  return l.M <= kLinearDecodeRows ? 0 : product_workspace(l.M, l.N, l.K);
}

size_t linear_backward_workspace_bytes(const moe_linear_t& l) {
  if (l.M == 0) return 0;
  return dpre_bytes(l) + part_bytes(l) +
         std::max(product_workspace(l.M, l.K, l.N), product_workspace(l.N, l.K, l.M));
}

hipError_t launch_linear(const moe_linear_t& l, const uint16_t* x, const uint16_t* w, const float* bias,
                         const void* residual, void* y, uint16_t* pre, void* workspace, hipStream_t st) {
  const Epilogue ep{bias, residual, y, pre, l.y_dtype == MOE_F32};
  if (l.M <= kLinearDecodeRows) return launch_linear_decode(l, x, w, ep, st);
  auto run = [&](auto act) {
    return launch_product<false, false, decltype(act)::value>(x, l.K, w, l.K, l.M, l.N, l.K, workspace, ep, st);
  };
  switch (l.act) {
    case MOE_ACT_RELU: return run(std::integral_constant<int, MOE_ACT_RELU>{});
    case MOE_ACT_SILU: return run(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU: return run(std::integral_constant<int, MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH: return run(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    default: return run(std::integral_constant<int, MOE_ACT_NONE>{});
  }
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
  void* partials = static_cast<uint8_t*>(workspace) + dpre_bytes(l) + part_bytes(l);
  if (e == hipSuccess && dx != nullptr)
    e = launch_product<false, true, MOE_ACT_NONE>(d, l.N, w, l.K, l.M, l.K, l.N, partials,
                                                  Epilogue{nullptr, nullptr, dx, nullptr, false}, st);
  if (e == hipSuccess && dw != nullptr)
    e = launch_product<true, true, MOE_ACT_NONE>(d, l.N, x, l.K, l.N, l.K, l.M, partials,
                                                 Epilogue{nullptr, nullptr, dw, nullptr, false}, st);
  return e;
}

}  // namespace moe
