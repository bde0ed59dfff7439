// Dense product for a few rows (decode): weight streaming.
//
// y = act(x w^T + bias) + residual with at most 32 rows reads w once and does
// little else, so the weight stream bounds it.  A workgroup owns CH output
// channels of RW rows and its W wavefronts share the contraction: wavefront v takes
// stages v, v + W, ... of 128 terms.  A stage's CH x 256 bytes come in the wide
// pattern (4 rows x 256 contiguous bytes per load, non-temporal: read once), D stages in
// flight in registers, go through the wavefront's own LDS tile (16-byte chunks
// XOR-swizzled by row; LDS operations of one wavefront execute in order, so no
// barrier) and come back in the v_mfma_f32_16x16x32_bf16 layout.  The rows of x
// (L2-resident) go the same way: read in the layout of the products instead, 16
// rows of 64 bytes a load, 32 rows took 31 us for 26 (MI355X, 14336 x 4096).  At
// the end the wavefronts' accumulators meet in LDS and are summed in wavefront
// order, 8 channels of a row to a lane.  Bound by the weight stream: 1 row, 14336
// x 4096: 21.2 us, 5.5 TB/s; few channels by what one CU takes in.
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "lds_stream.hpp"

namespace moe {
namespace {

constexpr int kStage = 128;                     // terms per stage
constexpr int kRowBytes = kStage * 2;

// Blocks of fewer than 16 channels or rows use that part of the 16 x 16 products.
template <int ACT, int RW, int CH, int W, int D>
__global__ __launch_bounds__(W * kWave) void linear_decode_kernel(const uint16_t* __restrict__ x,
                                                                  const uint16_t* __restrict__ w, int M, int N, int K,
                                                                  int row_blocks, const Epilogue ep) {
  constexpr int CG = (CH + 15) / 16, NT = (RW + 15) / 16;          // 16 x 16 products
  constexpr int WL = CH / 4, XL = RW / 4;                          // loads of a stage
  static_assert(CH % 8 == 0 && RW % 4 == 0 && (CH & (CH - 1)) == 0 && (RW & (RW - 1)) == 0, "whole loads and stores");
  static_assert(CG * RW * 16 * 4 <= (CH + RW) * kRowBytes, "the accumulators fit the tile");
  __shared__ __attribute__((aligned(16))) uint8_t lds[W][(CH + RW) * kRowBytes];
  const int block = xcd_remap(blockIdx.x, gridDim.x);           // a contiguous eighth of the channels per XCD
  const int c0 = block / row_blocks * CH, r0 = block % row_blocks * RW;
  if (c0 >= N) return;                                          // the whole workgroup
  const int lane = threadIdx.x & 63, v = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  uint8_t *tile = lds[v], *xtile = tile + CH * kRowBytes;
  // stage loads: lane (lrow, lch) takes chunk lch of rows lrow, lrow + 4, ...
  const int lrow = lane >> 4, lch = lane & 15;
  const int stages = (K + kStage - 1) / kStage;
  // descriptors bounded to the channels and rows there are: what lies past them
  // loads as zero; a chunk past the end of a row is sent past the descriptor
  const int rows = min(RW, M - r0);
  const __amdgpu_buffer_rsrc_t dw =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(w + (int64_t)c0 * K), 0, min(CH, N - c0) * K * 2, kRawBufferFlags);
  const __amdgpu_buffer_rsrc_t dx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x + (int64_t)r0 * K), 0, rows * K * 2, kRawBufferFlags);
  const int off = lrow * K * 2 + lch * 16;
  constexpr int kPast = (int)0x80000000u, kStream = 2;             // kStream: non-temporal, read once

  u32x4_t wv[D][WL], xv[D][XL];
  auto fetch = [&](u32x4_t (&wd)[WL], u32x4_t (&xd)[XL], int st) __attribute__((always_inline)) {
    const int k0 = st * kStage;
    const int wpast = k0 + lch * 8 < K ? 0 : kPast;
#pragma unroll
    for (int i = 0; i < WL; ++i)
      wd[i] = __builtin_amdgcn_raw_buffer_load_b128(dw, (off + i * 4 * K * 2) | wpast, k0 * 2, kStream);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      xd[i] = __builtin_amdgcn_raw_buffer_load_b128(dx, (off + i * 4 * K * 2) | wpast, k0 * 2, 0);
  };
  f32x4_t acc[CG][NT];
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[c][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto consume = [&](const u32x4_t (&wd)[WL], const u32x4_t (&xd)[XL]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int row = i * 4 + lrow;
      *reinterpret_cast<u32x4_t*>(tile + row * kRowBytes + ((lch ^ (row & 15)) << 4)) = wd[i];
    }
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int row = i * 4 + lrow;
      *reinterpret_cast<u32x4_t*>(xtile + row * kRowBytes + ((lch ^ (row & 15)) << 4)) = xd[i];
    }
    // (a block of fewer than 16 rows is read again for the others, whose products nobody looks at)
    auto read = [&](const uint8_t* t, int row, int j) __attribute__((always_inline)) {
      return *reinterpret_cast<const uint4*>(t + row * kRowBytes + (((4 * j + g) ^ (row & 15)) << 4));
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 xs[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) xs[n] = read(xtile, (n * 16 + r) & (RW - 1), j);
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        const uint4 a = read(tile, (c * 16 + r) & (CH - 1), j);
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
  // lane (r, g): row n 16 + r, channels 16 c + 4 g .. + 3; kept as [c][row][16]
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n * 16 + r < RW && 4 * g < CH)
        *reinterpret_cast<float4*>(tile + ((c * RW + n * 16 + r) * 16 + 4 * g) * 4) =
            make_float4(acc[c][n][0], acc[c][n][1], acc[c][n][2], acc[c][n][3]);
  __syncthreads();
  for (int o = threadIdx.x; o < rows * (CH / 8); o += W * kWave) {
    const int t = o / (CH / 8), q = o % (CH / 8), c = c0 + q * 8;
    if (c >= N) continue;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float p[8];
      load8f(reinterpret_cast<const float*>(lds[i]) + ((q >> 1) * RW + t) * 16 + (q & 1) * 8, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += p[k];
    }
    ep.store8<ACT>(r0 + t, c, N, sum);
  }
}

template <int ACT>
hipError_t launch_act(const moe_linear_t& l, const DecodeBlock& b, const uint16_t* x, const uint16_t* w,
                      const Epilogue& ep, hipStream_t st) {
  auto run = [&](auto kernel, int rw, int ch, int waves) {
    const int rb = (l.M + rw - 1) / rw, blocks = (l.N + ch - 1) / ch * rb;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((blocks + 7) / 8 * 8)), dim3(waves * kWave), 0, st, x, w, l.M, l.N, l.K, rb, ep);
    return hipGetLastError();
  };
  if (b.rows == 4) return run(linear_decode_kernel<ACT, 4, 8, 8, 2>, 4, 8, 8);
  if (b.rows == 8) return run(linear_decode_kernel<ACT, 8, 8, 8, 2>, 8, 8, 8);
  if (b.rows == 16) return run(linear_decode_kernel<ACT, 16, 16, 8, 1>, 16, 16, 8);
  if (b.channels == 32) return run(linear_decode_kernel<ACT, 32, 32, 4, 2>, 32, 32, 4);
  return run(linear_decode_kernel<ACT, 32, 16, 8, 1>, 32, 16, 8);
}

}  // namespace

hipError_t launch_linear_decode(const moe_linear_t& l, const DecodeBlock& block, const uint16_t* x, const uint16_t* w,
                                const Epilogue& ep, hipStream_t st) {
  switch (l.act) {
    case MOE_ACT_RELU: return launch_act<MOE_ACT_RELU>(l, block, x, w, ep, st);
    case MOE_ACT_SILU: return launch_act<MOE_ACT_SILU>(l, block, x, w, ep, st);
    case MOE_ACT_GELU: return launch_act<MOE_ACT_GELU>(l, block, x, w, ep, st);
    case MOE_ACT_GELU_TANH: return launch_act<MOE_ACT_GELU_TANH>(l, block, x, w, ep, st);
    default: return launch_act<MOE_ACT_NONE>(l, block, x, w, ep, st);
  }
}

}  // namespace moe
