// Products of a few rows with streamed weights (decode), shared by the dense product
// and the feed-forward block.
//
// A workgroup owns CH output channels of RW rows and its W wavefronts share the
// contraction: wavefront v takes stages v, v + W, ... of 128 terms.  A stage's CH x 256
// bytes come in the wide pattern (4 rows x 256 contiguous bytes per load, non-temporal:
// read once), D stages in flight in registers, go through the wavefront's own LDS tile
// (16-byte chunks XOR-swizzled by row; LDS operations of one wavefront execute in order,
// so no barrier) and come back in the v_mfma_f32_16x16x32_bf16 layout.  The rows of x
// (L2-resident) go the same way.
//
// PAIR: of each 16 channels the first 8 are w's and the last 8 w2's, the same 8 of both.
#pragma once
#include "device_common.hpp"
#include "lds_stream.hpp"
#include "linear_epilogue.hpp"

namespace moe {

constexpr int kStage = 128;                     // terms per stage
constexpr int kRowBytes = kStage * 2;

// Each wavefront's tile; afterwards its accumulators, as [c][row][16] for the channels'
// blocks c of 16.
template <int RW, int CH, int W>
struct StreamTiles {
  static_assert(CH % 8 == 0 && RW % 4 == 0 && (CH & (CH - 1)) == 0 && (RW & (RW - 1)) == 0, "whole loads and stores");
  static_assert((CH + 15) / 16 * RW * 16 * 4 <= (CH + RW) * kRowBytes, "the accumulators fit the tile");
  __attribute__((aligned(16))) uint8_t lds[W][(CH + RW) * kRowBytes];

  // Channels 8 q .. 8 q + 7 of row t, summed over the wavefronts in order.
  __device__ __forceinline__ void sum(int t, int q, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float p[8];
      load8f(reinterpret_cast<const float*>(lds[i]) + ((q >> 1) * RW + t) * 16 + (q & 1) * 8, p);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += p[k];
    }
  }
};

// x: the block's `rows` rows; w (and w2): its first channel, `channels` of them there.  Ends with a barrier.
// Blocks of fewer than 16 channels or rows use that part of the 16 x 16 products.
template <int RW, int CH, int W, int D, bool PAIR>
__device__ __forceinline__ void stream_products(StreamTiles<RW, CH, W>& tiles, const uint16_t* x, int rows,
                                                const uint16_t* w, const uint16_t* w2, int channels, int K) {
  constexpr int CG = (CH + 15) / 16, NT = (RW + 15) / 16;          // 16 x 16 products
  constexpr int WL = CH / 4, XL = RW / 4;                          // loads of a stage
  const int lane = threadIdx.x & 63, v = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  uint8_t *tile = tiles.lds[v], *xtile = tile + CH * kRowBytes;
  // stage loads: lane (lrow, lch) takes chunk lch of rows lrow, lrow + 4, ...
  const int lrow = lane >> 4, lch = lane & 15;
  const int stages = (K + kStage - 1) / kStage;
  // descriptors bounded to the channels and rows there are: what lies past them
  // loads as zero; a chunk past the end of a row is sent past the descriptor
  const __amdgpu_buffer_rsrc_t dw =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(w), 0, channels * K * 2, kRawBufferFlags);
  const __amdgpu_buffer_rsrc_t dw2 =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(w2), 0, channels * K * 2, kRawBufferFlags);
  const __amdgpu_buffer_rsrc_t dx =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(x), 0, rows * K * 2, kRawBufferFlags);
  const int off = lrow * K * 2 + lch * 16;
  constexpr int kPast = (int)0x80000000u, kStream = 2;             // kStream: non-temporal, read once

  u32x4_t wv[D][WL], xv[D][XL];
  auto fetch = [&](u32x4_t (&wd)[WL], u32x4_t (&xd)[XL], int st) __attribute__((always_inline)) {
    const int k0 = st * kStage;
    const int wpast = k0 + lch * 8 < K ? 0 : kPast;
#pragma unroll
    for (int i = 0; i < WL; ++i)
      // (PAIR: loads 4 n and 4 n + 1 bring w's 8 channels, the other two w2's)
      wd[i] = __builtin_amdgcn_raw_buffer_load_b128(PAIR && (i & 2) ? dw2 : dw,
                                                    (off + (PAIR ? (i >> 2) * 2 + (i & 1) : i) * 4 * K * 2) | wpast, k0 * 2,
                                                    kStream);
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
}

}  // namespace moe
