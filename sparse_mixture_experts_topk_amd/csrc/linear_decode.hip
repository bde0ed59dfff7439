// Dense product for a few rows (decode): weight streaming.
//
// y = act(x w^T + bias) + residual with at most 32 rows reads w once and does
// little else, so the weight stream bounds it (stream_products.hpp).  The rows of x
// go through LDS like the weights: read in the layout of the products instead, 16
// rows of 64 bytes a load, 32 rows took 31 us for 26 (MI355X, 14336 x 4096).  At
// the end the wavefronts' accumulators meet in LDS and are summed in wavefront
// order, 8 channels of a row to a lane.  Bound by the weight stream: 1 row, 14336
// x 4096: 21.2 us, 5.5 TB/s; few channels by what one CU takes in.
#include "device_common.hpp"
#include "launch.hpp"
#include "linear_epilogue.hpp"
#include "stream_products.hpp"

namespace moe {
namespace {

// Blocks of fewer than 16 channels or rows use that part of the 16 x 16 products.
template <int ACT, int RW, int CH, int W, int D>
__global__ __launch_bounds__(W * kWave) void linear_decode_kernel(const uint16_t* __restrict__ x,
                                                                  const uint16_t* __restrict__ w, int M, int N, int K,
                                                                  int row_blocks, const Epilogue ep) {
  __shared__ StreamTiles<RW, CH, W> tiles;
  const int block = xcd_remap(blockIdx.x, gridDim.x);           // a contiguous eighth of the channels per XCD
  const int c0 = block / row_blocks * CH, r0 = block % row_blocks * RW;
  if (c0 >= N) return;                                          // the whole workgroup
  const int rows = min(RW, M - r0);
  stream_products<RW, CH, W, D, false>(tiles, x + (int64_t)r0 * K, rows, w + (int64_t)c0 * K, nullptr, min(CH, N - c0), K);
  for (int o = threadIdx.x; o < rows * (CH / 8); o += W * kWave) {
    const int t = o / (CH / 8), q = o % (CH / 8), c = c0 + q * 8;
    if (c >= N) continue;
    float sum[8];
    tiles.sum(t, q, sum);
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
