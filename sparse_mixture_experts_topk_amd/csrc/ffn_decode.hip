// Gate/up product of the feed-forward block for a few dense rows (decode): both
// weights are streamed once (stream_products.hpp), 8 channels of w1 and the same 8 of w3
// to each 16 x 16 product, so that a workgroup ends with g and u of its channels and
// stores h.  Bound by the weight stream.
#include "device_common.hpp"
#include "ffn_groups.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "stream_products.hpp"

namespace moe {
namespace {

struct FfnDecodeArgs {
  const uint16_t *x, *w1, *w3;
  const int32_t* offsets;        // NULL, or the bounds of the one group
  int M, F, K, row_blocks, act;
  uint16_t *h, *g, *u;
};

// CH / 2 channels of each weight.
template <int RW, int CH, int W, int D>
__global__ __launch_bounds__(W * kWave) void ffn_decode_kernel(const FfnDecodeArgs a) {
  __shared__ StreamTiles<RW, CH, W> tiles;
  const int block = xcd_remap(blockIdx.x, gridDim.x);           // a contiguous eighth of the channels per XCD
  const int c0 = block / a.row_blocks * (CH / 2);
  if (c0 >= a.F) return;                                        // the whole workgroup
  int first = 0, end = a.M;
  if (a.offsets != nullptr) {
    first = min(max(a.offsets[0], 0), a.M);
    end = max(min(a.offsets[1], a.M), first);
  }
  const int r0 = first + block % a.row_blocks * RW, rows = min(RW, end - r0);
  if (rows <= 0) return;
  const int64_t w = (int64_t)c0 * a.K;
  stream_products<RW, CH, W, D, true>(tiles, a.x + (int64_t)r0 * a.K, rows, a.w1 + w, a.w3 + w, min(CH / 2, a.F - c0), a.K);
  for (int o = threadIdx.x; o < rows * (CH / 16); o += W * kWave) {
    const int t = o / (CH / 16), q = o % (CH / 16), c = c0 + q * 8;
    if (c >= a.F) continue;
    float g[8], u[8];
    tiles.sum(t, 2 * q, g);
    tiles.sum(t, 2 * q + 1, u);
    const int64_t at = (int64_t)(r0 + t) * a.F + c;
    if (a.g != nullptr) {
      *reinterpret_cast<uint4*>(a.g + at) = pack8(g);
      *reinterpret_cast<uint4*>(a.u + at) = pack8(u);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = act_value<false>(g[k], a.act) * u[k];
    *reinterpret_cast<uint4*>(a.h + at) = pack8(g);
  }
}

}  // namespace

hipError_t launch_ffn_decode(const moe_ffn_t& f, const DecodeBlock& b, const FfnTensors<uint16_t>& t, hipStream_t st) {
  FfnDecodeArgs a{t.x, t.w1, t.w3, t.offsets, f.M, f.d_ff, f.d_model, (f.M + b.rows - 1) / b.rows, f.act,
                  t.h_out, t.g_out, t.u_out};
  const int blocks = (f.d_ff + b.channels / 2 - 1) / (b.channels / 2) * a.row_blocks;
  auto run = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((blocks + 7) / 8 * 8)), dim3(waves * kWave), 0, st, a);
    return hipGetLastError();
  };
  if (b.rows == 4) return run(ffn_decode_kernel<4, 16, 8, 2>, 8);
  if (b.rows == 8) return run(ffn_decode_kernel<8, 16, 8, 2>, 8);
  if (b.rows == 16) return run(ffn_decode_kernel<16, 16, 8, 1>, 8);
  if (b.channels == 32) return run(ffn_decode_kernel<32, 32, 4, 2>, 4);
  return run(ffn_decode_kernel<32, 16, 8, 1>, 8);
}

}  // namespace moe
