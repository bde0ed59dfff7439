// Dense product for a few rows (decode): weight streaming.
//
// y = act(x w^T + bias) + residual with M <= 16 NT rows reads w once and does
// little else, so the weight stream bounds it.  A workgroup owns 16 output
// channels and its W wavefronts share the contraction: wavefront v takes stages
// v, v + W, ... of 128 terms.  A stage's 16 x 256 bytes come in the wide pattern
// (4 rows x 256 contiguous bytes per load, non-temporal: read once), D stages in
// flight in registers, go through the wavefront's own LDS tile (16-byte chunks
// XOR-swizzled by row; LDS operations of one wavefront execute in order, so no
// barrier) and come back in the v_mfma_f32_16x16x32_bf16 layout.  The rows of x
// (L2-resident) go the same way: read in the layout of the products instead, 16
// rows of 64 bytes a load, 32 rows took 31 us for 26 (MI355X, 14336 x 4096).  At
// the end the wavefronts' accumulators meet in LDS and are summed in wavefront
// order, 8 channels of a row to a lane.  Bound by the weight stream: 1 row, 14336
// x 4096: 21.2 us, 5.5 TB/s; few channels by latency (16 rows, 256 x 4096: 6.8 us).
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "lds_stream.hpp"

namespace moe {
namespace {

constexpr int kStage = 128;                     // terms per stage
constexpr int kTileBytes = 16 * kStage * 2;     // one wavefront's LDS tile

template <int ACT, int NT, int CG, int W, int D>
__global__ __launch_bounds__(W * kWave) void linear_decode_kernel(const uint16_t* __restrict__ x,
                                                                  const uint16_t* __restrict__ w, int M, int N, int K,
                                                                  const Epilogue ep) {
  static_assert(NT * 16 * 16 * 4 <= kTileBytes, "the accumulators fit the tile");
  __shared__ __attribute__((aligned(16))) uint8_t lds[W][(CG + NT) * kTileBytes];
  const int c0 = xcd_remap(blockIdx.x, gridDim.x) * (16 * CG);  // a contiguous eighth of the channels per XCD
  if (c0 >= N) return;                                          // the whole workgroup
  const int lane = threadIdx.x & 63, v = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  uint8_t* tile = lds[v];
  // stage loads: lane (lrow, lch) takes chunk lch of rows lrow, lrow + 4, ...; channels past N repeat the last
  const int lrow = lane >> 4, lch = lane & 15;
  const int stages = (K + kStage - 1) / kStage;
  // descriptors bounded to the channels and rows there are: what lies past them
  // loads as zero; a chunk past the end of a row is sent past the descriptor
  const __amdgpu_buffer_rsrc_t dw =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(w + (int64_t)c0 * K), 0, min(16 * CG, N - c0) * K * 2, kRawBufferFlags);
  const __amdgpu_buffer_rsrc_t dx = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x), 0, M * K * 2, kRawBufferFlags);
  const int off = lrow * K * 2 + lch * 16;
  constexpr int kPast = (int)0x80000000u, kStream = 2;             // kStream: non-temporal, read once

  u32x4_t wv[D][CG * 4], xv[D][NT * 4];
  auto fetch = [&](u32x4_t (&wd)[CG * 4], u32x4_t (&xd)[NT * 4], int st) __attribute__((always_inline)) {
    const int k0 = st * kStage;
    const int wpast = k0 + lch * 8 < K ? 0 : kPast;
#pragma unroll
    for (int i = 0; i < CG * 4; ++i)
      wd[i] = __builtin_amdgcn_raw_buffer_load_b128(dw, (off + i * 4 * K * 2) | wpast, k0 * 2, kStream);
#pragma unroll
    for (int i = 0; i < NT * 4; ++i)
      xd[i] = __builtin_amdgcn_raw_buffer_load_b128(dx, (off + i * 4 * K * 2) | wpast, k0 * 2, 0);
  };
  f32x4_t acc[CG][NT];
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[c][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto consume = [&](const u32x4_t (&wd)[CG * 4], const u32x4_t (&xd)[NT * 4]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CG * 4; ++i) {
      const int row = i * 4 + lrow;
      *reinterpret_cast<u32x4_t*>(tile + row * (kStage * 2) + ((lch ^ (row & 15)) << 4)) = wd[i];
    }
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) {
      const int row = i * 4 + lrow;
      *reinterpret_cast<u32x4_t*>(tile + CG * kTileBytes + row * (kStage * 2) + ((lch ^ (row & 15)) << 4)) = xd[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 xs[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        xs[n] = *reinterpret_cast<const uint4*>(tile + CG * kTileBytes + (n * 16 + r) * (kStage * 2) + (((4 * j + g) ^ r) << 4));
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        const uint4 a = *reinterpret_cast<const uint4*>(tile + (c * 16 + r) * (kStage * 2) + (((4 * j + g) ^ r) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[c][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(xs[n]), acc[c][n], 0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(wv[d], xv[d], v + d * W);      // past the end: zeros, nothing read
  for (int st = v; st < stages; st += D * W) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      consume(wv[d], xv[d]);
      fetch(wv[d], xv[d], st + (d + D) * W);
    }
  }
  // lane (r, g): row n 16 + r, channels 16 c + 4 g .. + 3
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float4*>(tile + c * kTileBytes + ((n * 16 + r) * 16 + 4 * g) * 4) =
          make_float4(acc[c][n][0], acc[c][n][1], acc[c][n][2], acc[c][n][3]);
  __syncthreads();
  for (int o = threadIdx.x; o < M * 2 * CG; o += W * kWave) {
    const int t = o / (2 * CG), q = o % (2 * CG), c = c0 + q * 8;
    if (c >= N) continue;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float p[8];
      load8f(reinterpret_cast<const float*>(lds[i] + (q >> 1) * kTileBytes) + t * 16 + (q & 1) * 8, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += p[k];
    }
    ep.store8<ACT>(t, c, N, sum);
  }
}

// One block of 16 channels and 8 wavefronts per workgroup, one stage in flight
// each.  Two blocks of rows leave LDS for one such workgroup per CU: where there
// are more channels than one round of them takes, 4 wavefronts on two blocks of
// channels, two workgroups per CU, share each read of x twice.  MI355X, us, wide
// against narrow: 32 rows of 4096 terms, N 4096 13.3 / 11.6, N 6144 14.3 / 18.7, N
// 14336 25.8 / 35.3; with 16 rows N 12288 21.8 / 19.3, N 14336 23.1 / 24.0.  16
// wavefronts or two stages in flight gain nothing (16 rows, N 4096: 10.2, 9.6 / 9.2).
template <int ACT, int NT>
hipError_t launch_act(const moe_linear_t& l, const uint16_t* x, const uint16_t* w, const Epilogue& ep,
                      hipStream_t st) {
  auto run = [&](auto kernel, int cg, int waves) {
    const int groups = (l.N + 16 * cg - 1) / (16 * cg);
    hipLaunchKernelGGL(kernel, dim3((unsigned)((groups + 7) / 8 * 8)), dim3(waves * kWave), 0, st, x, w, l.M, l.N, l.K, ep);
    return hipGetLastError();
  };
  if constexpr (NT == 2) {
    if ((l.N + 15) / 16 > device_cu_count()) return run(linear_decode_kernel<ACT, NT, 2, 4, 2>, 2, 4);
  }
  return run(linear_decode_kernel<ACT, NT, 1, 8, 1>, 1, 8);
}

template <int ACT>
hipError_t launch_rows(const moe_linear_t& l, const uint16_t* x, const uint16_t* w, const Epilogue& ep,
                       hipStream_t st) {
  if (l.M <= 16) return launch_act<ACT, 1>(l, x, w, ep, st);
  return launch_act<ACT, 2>(l, x, w, ep, st);
}

}  // namespace

hipError_t launch_linear_decode(const moe_linear_t& l, const uint16_t* x, const uint16_t* w, const Epilogue& ep,
                                hipStream_t st) {
  switch (l.act) {
    case MOE_ACT_RELU: return launch_rows<MOE_ACT_RELU>(l, x, w, ep, st);
    case MOE_ACT_SILU: return launch_rows<MOE_ACT_SILU>(l, x, w, ep, st);
    case MOE_ACT_GELU: return launch_rows<MOE_ACT_GELU>(l, x, w, ep, st);
    case MOE_ACT_GELU_TANH: return launch_rows<MOE_ACT_GELU_TANH>(l, x, w, ep, st);
    default: return launch_rows<MOE_ACT_NONE>(l, x, w, ep, st);
  }
}

}  // namespace moe
